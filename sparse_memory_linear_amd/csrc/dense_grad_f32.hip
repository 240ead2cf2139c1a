// dense_grad_f32.hip -- the dense recurrence's passes for the gradients, over fp32 rows.
#include "dense_pass.h"

namespace sdm {

hipError_t launch_dense_grads_f32(const DenseArgs& q, const DenseArgs& k, const DenseArgs& v, hipStream_t st) {
    return dense_grads<3>(q, k, v, st);
}

}  // namespace sdm
