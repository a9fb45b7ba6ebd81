// Causal attention of packed queries (packed_att.cuh) without score options.
#include "packed_att.cuh"

namespace ha {

int packed_key_tile(bool f32_out) { return f32_out ? 64 : 128; }

cudaError_t launch_packed_att(const PackedParams& p, const PackedMaps& m, int d, bool f32_out, int grid, bool merge,
                              cudaStream_t st) {
    return launch<kPlain>(p, m, d, f32_out, grid, merge, st);
}

}  // namespace ha
