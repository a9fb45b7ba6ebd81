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

// n / d for 0 <= n < 2^31 and d >= 1 as a product: with 2^k < d <= 2^(k + 1) and m = ceil(2^(32 + k) / d),
// m d exceeds 2^(32 + k) by less than d, so m n / 2^(32 + k) exceeds n / d by less than 1 / d.
struct Quotient {
    uint32_t m;
    int k;  // -1: d is 1
    static Quotient of(uint32_t d) {
        int k = -1;
        while (((uint64_t)1 << (k + 1)) < d) ++k;
        return Quotient{k < 0 ? 0u : (uint32_t)((((uint64_t)1 << (32 + k)) + d - 1u) / d), k};
    }
    HA_HD int operator()(int n) const {
        return k < 0 ? n : (int)((uint32_t)((uint64_t)(uint32_t)n * m >> 32) >> k);
    }
};

// The keys and key tiles (2^K keys) of a row of items under score options: t2 new tokens to an item;
// token t of nq, whose position is base + t, sees the keys max(first, base + t + 1 - window) <= j <
// max(base + t + 1, prefix) below nk = base + nq (window 0: none; first and prefix lie within [0, nk]).
// Both ends grow with the item, each from where it leaves a constant, so the work of a row of items
// is two constants and two sums in closed form.
template <int K>
struct MaskedItems {
    int base, nq, first, prefix, window, t2;
    Quotient per;  // by t2
    HA_HD static int least(int a, int b) { return a < b ? a : b; }
    HA_HD static int most(int a, int b) { return a > b ? a : b; }
    HA_HD static int tiles_of(int keys) { return (keys + (1 << K) - 1) >> K; }
    // end of the keys that the first `upto` tokens see
    HA_HD int end(int upto) const { return most(base + least(upto, nq), prefix); }
    // the first key that token t sees, if it sees any
    HA_HD int begin(int t) const { return window > 0 ? most(first, base + t + 1 - window) : first; }
    // An item's first tile (0 where it sees no key) and its tiles (then 1, so that its rows are written).
    HA_HD bool none(int qt) const { return begin(qt * t2) >= end((qt + 1) * t2); }
    HA_HD int begin_tile(int qt) const { return none(qt) ? 0 : begin(qt * t2) >> K; }
    HA_HD int tiles(int qt) const { return none(qt) ? 1 : tiles_of(end((qt + 1) * t2)) - (begin(qt * t2) >> K); }
    // tiles of the items 0 .. qt - 1, all of t2 tokens
    HA_HD uint32_t tiles_before(int qt, const TileSums<K>& sums, const uint16_t* before) const {
        if (qt == 0) return 0;
        // items 0 .. z - 1 see no key: they end at or before `first`
        const int z = prefix > first || base > first ? 0 : least(qt, per(first - base));
        // items z .. e - 1 end with the prefix
        const int e = base > prefix ? z : least(qt, most(z, per(prefix - base)));
        uint32_t c = (uint32_t)z + (uint32_t)(e - z) * (uint32_t)tiles_of(prefix);
        if (qt > e) c += sums.sum((uint32_t)(qt - e), (uint32_t)(base + (e + 1) * t2 + (1 << K) - 1), before);
        // items z .. b - 1 begin at `first`
        int b = qt;
        if (window > 0) {
            const int w = base + 1 - window;
            b = w > first ? z : least(qt, most(z, per(first - w) + 1));
            if (qt > b) c -= sums.sum((uint32_t)(qt - b), (uint32_t)(w + b * t2), before);
        }
        return c - (uint32_t)(b - z) * (uint32_t)(first >> K);
    }
};

// The references that rows of capped scores over up to `keys` keys may keep (scores within +-cap, in powers of 2). With
// a reference r in [low, high] a weight 2^{score - r} is at most 2^(cap - low): as many of them as there are
// keys times values below 2^20 stay below 2^125 (2^24 keys: 2^124). And it is at least 2^-kDown, whose
// products with values are sums of the smallest numbers that the accumulators hold, multiples of 2^-149: a
// value from 2^-40 on keeps 24 bits beside it, three parts of a weight included.
struct CapRange {
    static constexpr int kUp = 80, kAll = 105, kDown = 85;
    double low, high;
    HA_HD static CapRange of(double cap, int keys) {
        int log2 = 0;  // of the keys, rounded up
        while (((int64_t)1 << log2) < keys) ++log2;
        const int up = kAll - log2 < kUp ? kAll - log2 : kUp;
        return CapRange{cap - up, kDown - cap};
    }
    HA_HD bool fits() const { return low <= high; }
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
