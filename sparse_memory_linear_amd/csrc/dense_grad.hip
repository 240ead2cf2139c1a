// dense_grad.hip -- the dense recurrence's passes that mix bf16 rows with the fp32 rows of dy (dq, dk, dv).
#include "dense_pass.h"

namespace sdm {

hipError_t launch_dense_xi32(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<DENSE_CHUNK_F32, 3, 1, 1, true, true>(a, st); }
hipError_t launch_dense_kap32(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<DENSE_CHUNK_F32, 1, 3, 1, true, true>(a, st); }
hipError_t launch_dense_omg32(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<DENSE_CHUNK_F32, 1, 1, 3, true, false>(a, st); }
hipError_t launch_dense_omg32_state(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<DENSE_CHUNK, 1, 1, 3, false, false>(a, st); }

}  // namespace sdm
