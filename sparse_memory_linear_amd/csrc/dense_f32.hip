// dense_f32.hip -- the dense recurrence's passes over fp32 rows: y, and the segments' own states.
#include "dense_pass.h"

namespace sdm {

hipError_t launch_dense_y_f32(const DenseArgs& a, hipStream_t st) { return dense_y<3, 3, 3>(a, st); }
hipError_t launch_dense_s_f32(const DenseArgs& a, hipStream_t st) { return dense_s<3, 3>(a, st); }
hipError_t launch_dense_sg_f32(const DenseArgs& s, const DenseArgs& g, hipStream_t st) { return dense_sg<3, 3, 3>(s, g, st); }

}  // namespace sdm
