// The order of the products of a segment of k_packed_att whose S and P have three places
// (head dim 64): which stream and key tile product k belongs to. One function for the warp that
// issues the products and the warps that wait for them; plain C++, so that a host test
// can go through all segments.
#pragma once

#ifdef __CUDACC__
#define HA_HD __host__ __device__ __forceinline__
#else
#define HA_HD inline
#endif

namespace ha {

// One row tile: the key tiles in turn, even ones stream 0's. Two: key tile by key tile, row
// tile 0 (the first e0 key tiles only) before row tile 1 (all nt, e0 <= nt).
struct Products {
    int e0, nt;
    bool one;
    HA_HD int count() const { return one ? nt : e0 + nt; }
    HA_HD int tiles(int t) const { return one ? (nt + 1 - t) >> 1 : (t == 0 ? e0 : nt); }
    // the last product of its key tile
    HA_HD bool last_of_tile(int k) const { return one || k >= 2 * e0 || (k & 1) != 0; }
    HA_HD int stream(int k, bool last) const { return one ? k & 1 : (last ? 1 : 0); }  // last: last_of_tile(k)
    // product of stream t's tile i
    HA_HD int of(int t, int i) const { return one ? 2 * i + t : (i < e0 ? 2 * i + t : e0 + i); }
    // A later product of the segment uses the place of stream t's last one: only row tile 0 can end
    // three products ahead.
    HA_HD bool lapped(int t) const { return !one && t == 0 && nt > e0 + 1; }
};

}  // namespace ha
