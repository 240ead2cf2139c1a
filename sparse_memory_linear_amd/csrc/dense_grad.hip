// dense_grad.hip -- the dense recurrence's passes for the gradients, over bf16 rows (dy's are fp32).
#include "dense_pass.h"

namespace sdm {

hipError_t launch_dense_grads(const DenseArgs& q, const DenseArgs& k, const DenseArgs& v, hipStream_t st) {
    return dense_grads<1>(q, k, v, st);
}

}  // namespace sdm
