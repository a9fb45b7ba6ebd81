// Attention of packed queries (packed_att.cuh) with capped scores.
#include "packed_att.cuh"

namespace ha {

cudaError_t launch_packed_att_capped(const PackedParamsEx& p, const PackedMaps& m, int d, bool f32_out, int grid, bool merge,
                                     cudaStream_t st) {
    if (d == 128 && !f32_out && p.long_items) return launch_128<kCappedLong>(p, m, grid, merge, st);
    return launch<kCapped>(p, m, d, f32_out, grid, merge, st);
}

}  // namespace ha
