// dense_bf16.hip -- the dense recurrence's passes over bf16 rows (the forward).
#include "dense_pass.h"

namespace sdm {

hipError_t launch_dense_bf16(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<DENSE_CHUNK, 1, 1, 1, true, false>(a, st); }
hipError_t launch_dense_bf16_state(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<DENSE_CHUNK, 1, 1, 1, false, false>(a, st); }

}  // namespace sdm
