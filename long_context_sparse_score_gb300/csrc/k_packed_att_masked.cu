// Attention of packed queries (packed_att.cuh) with masks alone (a window, a prefix, first keys), or another scale.
#include "packed_att.cuh"

namespace ha {

cudaError_t launch_packed_att_masked(const PackedParamsEx& p, const PackedMaps& m, int d, bool f32_out, int grid, bool merge,
                                     cudaStream_t st) {
    return launch<kMasked>(p, m, d, f32_out, grid, merge, st);
}

}  // namespace ha
