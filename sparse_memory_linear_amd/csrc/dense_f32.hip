// dense_f32.hip -- the dense recurrence's passes over fp32 rows: y, and the segments' own states S and G.
#include "dense_pass.h"

namespace sdm {

hipError_t launch_dense_y_f32(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<3, 3, 3, true, false, false>(a, st); }
hipError_t launch_dense_s_f32(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<3, 3, 3, false, false, false>(a, st); }
hipError_t launch_dense_g_f32(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<3, 3, 3, false, true, false>(a, st); }

}  // namespace sdm
