// dense_bf16.hip -- the dense recurrence's passes over bf16 rows: y, and the segments' own states S.
#include "dense_pass.h"

namespace sdm {

hipError_t launch_dense_y(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<1, 1, 1, true, false, false>(a, st); }
hipError_t launch_dense_s(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<1, 1, 1, false, false, false>(a, st); }

}  // namespace sdm
