// dense_grad_f32.hip -- the dense recurrence's passes over fp32 rows: the gradients.
#include "dense_pass.h"

namespace sdm {

hipError_t launch_dense_dq_f32(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<3, 3, 3, true, false, true>(a, st); }
hipError_t launch_dense_dk_f32(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<3, 3, 3, true, true, true>(a, st); }
hipError_t launch_dense_dv_f32(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<3, 3, 3, true, true, false>(a, st); }

}  // namespace sdm
