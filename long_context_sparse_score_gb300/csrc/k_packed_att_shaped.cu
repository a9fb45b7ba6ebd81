// Attention of packed queries (packed_att.cuh) with biased scores, or capped ones of any range.
#include "packed_att.cuh"

namespace ha {

cudaError_t launch_packed_att_shaped(const PackedParamsEx& p, const PackedMaps& m, int d, bool f32_out, int grid, bool merge,
                                     cudaStream_t st) {
    return launch<kShaped>(p, m, d, f32_out, grid, merge, st);
}

}  // namespace ha
