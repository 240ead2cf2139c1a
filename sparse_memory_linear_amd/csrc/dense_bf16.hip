// dense_bf16.hip -- the dense recurrence's passes over bf16 rows (dy's are fp32): y, and the segments' own states.
#include "dense_pass.h"

namespace sdm {

hipError_t launch_dense_y(const DenseArgs& a, hipStream_t st) { return dense_y<1, 1, 1>(a, st); }
hipError_t launch_dense_s(const DenseArgs& a, hipStream_t st) { return dense_s<1, 1>(a, st); }
hipError_t launch_dense_sg(const DenseArgs& s, const DenseArgs& g, hipStream_t st) { return dense_sg<1, 1, 3>(s, g, st); }

}  // namespace sdm
