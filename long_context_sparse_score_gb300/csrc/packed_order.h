// What the roles of k_packed_att agree on, in plain C++, so that a host test can go through it: the
// work of a row of items, and the order of a segment's products.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define HA_HD __host__ __device__ __forceinline__
#else
#define HA_HD inline
#endif

namespace ha {

// Key tiles of a row of items: sum over i < n of floor((a i + b) / 2^K), where item i sees
// a i + b - 2^K + 1 keys more than none (a: tokens of an item, at most 256 and even; the sum is below 2^32).
// The quotients add up to ((a n (n - 1) / 2 + b n) - R) / 2^K with R the sum of the remainders. With
// g = gcd(a, 2^K), the remainders of a i are g times those of (a / g) i modulo P = 2^K / g, which go
// through every value once in P items, and b only shifts where they begin: b mod 2^K = a s + (b mod g)
// modulo 2^K for s = (b / g) (a / g)^-1 modulo P. So R needs the sums over the first x < P <= 32 or 64
// remainders, which are the same for all sequences.
template <int K>
struct TileSums {
    static constexpr int kMost = 1 << (K - 1);  // entries of `before`: P is at most half a tile, as a is even
    uint32_t a;
    uint32_t lg, odd, inv;  // log2 g, a / g, its inverse modulo 2^12
    HA_HD explicit TileSums(uint32_t tokens) : a(tokens), lg(0) {
        while (lg < (uint32_t)K && ((a >> lg) & 1u) == 0u) ++lg;
        odd = a >> lg;
        inv = odd * (2u - odd * odd);        // modulo 64, as odd is its own inverse modulo 8
        inv = inv * (2u - odd * inv);
    }
    HA_HD uint32_t period() const { return (1u << K) >> lg; }
    HA_HD uint32_t remainder(uint32_t i) const { return (odd * i) & (period() - 1u); }
    // before[x]: remainder(0) + .. + remainder(x - 1)
    HA_HD uint32_t sum(uint32_t n, uint32_t b, const uint16_t* before) const {
        const uint32_t P = period(), s = ((b >> lg) * inv) & (P - 1u), e = s + n, turns = e >> (K - lg);
        const uint64_t R = (uint64_t)(b & ((1u << lg) - 1u)) * n +
                           (((uint64_t)turns * (P * (P - 1u) / 2u) + before[e & (P - 1u)] - before[s]) << lg);
        return (uint32_t)(((uint64_t)a * ((uint64_t)n * (n - 1u) / 2u) + (uint64_t)b * n - R) >> K);
    }
};

// The order of the products of a segment whose S and P have three places (head dim 64): which stream
// and key tile product k belongs to, for the warp that issues them and the warps that wait for them.
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
