// dense_grad.hip -- the dense recurrence's passes that mix bf16 rows with the fp32 rows of dy.
#include "dense_pass.h"

namespace sdm {

hipError_t launch_dense_dq(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<3, 1, 1, true, false, true>(a, st); }
hipError_t launch_dense_dk(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<1, 3, 1, true, true, true>(a, st); }
hipError_t launch_dense_dv(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<1, 1, 3, true, true, false>(a, st); }
hipError_t launch_dense_g(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<1, 1, 3, false, true, false>(a, st); }

}  // namespace sdm
