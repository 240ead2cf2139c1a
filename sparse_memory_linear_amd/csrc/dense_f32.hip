// dense_f32.hip -- the dense recurrence's passes over fp32 rows.
#include "dense_pass.h"

namespace sdm {

hipError_t launch_dense_f32(const DenseArgs& a, hipStream_t st) {
    return a.dot ? launch_dense_sized<DENSE_CHUNK_F32, 3, 3, 3, true, true>(a, st)
                 : launch_dense_sized<DENSE_CHUNK_F32, 3, 3, 3, true, false>(a, st);
}
hipError_t launch_dense_f32_state(const DenseArgs& a, hipStream_t st) { return launch_dense_sized<DENSE_CHUNK_F32, 3, 3, 3, false, false>(a, st); }

}  // namespace sdm
