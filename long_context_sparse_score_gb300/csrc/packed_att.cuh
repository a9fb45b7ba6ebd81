// Attention of packed queries: whole prompts (K and V packed like the queries) and
// chunks of new tokens over a paged cache; causal, or with score options (below).
//
// Row (token i of sequence s, query head h) with g = h / G attends to the keys
// j < L(i) = nk - nq + i + 1 of its sequence (nq new tokens, nk keys in all):
//   z_j = <q, K_j> / sqrt(d),  out = sum_j e^{z_j} V_j / sum_j e^{z_j},
//   lse = log sum_j e^{z_j}    (L(i) <= 0: out = 0, lse = -inf)
// (HashAttention: Semantic Sparsity for Faster Inference, Sec. 4 estimator with
// every visible token selected; lse as in Nectar, Eq. (3.1)).
//
// One pass over the keys with a running reference maximum m and mass l per row:
// S = Q K^T (tcgen05.mma, float32 accumulator in tensor memory), P = 2^{(S - m)
// log2(e)/sqrt(d)} rounded to bf16 in tensor memory, O += P V (P read as the
// MMA's A operand from tensor memory). O is rescaled only when a row's maximum
// grows by more than 2^8 over its reference: until then P <= 2^8, which costs
// neither range nor precision, as bf16 keeps its relative step. l is summed in
// float32 from the values before they are rounded.
// With a float32 output, P enters as three bf16 parts, each the rounding of what the
// earlier ones left (together all 24 bits of p), for three times the P V products;
// tiles are 64 keys, so that the parts fit beside and over S. The tensor cores'
// accumulator cuts off instead of rounding (measured: 2e-8 a step, 1.2e-5 of O after
// 3,500 keys), so a tile's O is added to float32 sums in registers.
//
// Rows: the G query heads of a KV head share its K and V, so a tile packs
// TQ = floor(128 / G) tokens x G heads (row = token * G + head). An item is
// (sequence, KV head, 2 TQ tokens): two tiles, one softmax warpgroup each, so
// that one tile's exponentials run under the other tile's products. An item of
// at most TQ tokens (decode) has one tile: its warpgroups take the even and the
// odd key tiles, each with its own m, l, O, which are joined at the end.
//
// Work is cut at key tiles, not at items: CTA c of P takes the tiles
// [c U / P, (c + 1) U / P) of all items in order, so any mix of lengths fills
// the GPU. A boundary close to an item's edge moves to it. Parts of an item that
// spans CTAs go to the workspace (unnormalised O, m, l) and k_packed_merge joins
// them, in order, so results do not depend on timing.
//
// Measured (graph replays; rates against cuBLAS's bf16 burst and a plain copy): a prompt of
// 16,384 tokens, 32/8 heads of 128: 1.33 to 1.37 ms, 1.65 PFLOP/s, 86 % (1.43 ms at the power cap);
// 24 prompts of 33 to 2,500: 330 to 334 us, 58 % (an item's start and end cost each CTA about
// 6,000 cycles, two tiles); 16,384 tokens at d 64: 1.10 ms, 52 % (bound by the softmax
// warps' latency, not by a unit); decode of 64 sequences of 1,000 to 16,000 keys: 345 us,
// 6.4 TB/s, 95 %; one token over 131,072 keys, float32 out: 108 us, 5.0 TB/s, 73 % (bound by
// the products: three for P V); 4 x 512 tokens over 20,000 to 32,000 keys: 574 us, 84 %.
//
// Score options (ha_score_opts) are kernels of their own (Mode), so that calls without them run the code
// that they ran before. With pos the row's position, z_j becomes cap tanh(scale <q, K_j> / cap) - slope
// |pos - j|, over max(first, pos - window + 1) <= j < max(pos + 1, prefix).
// - Masks leave a row one interval of keys whose ends grow with the row, so an item has one range of
//   key tiles, and their sum over a row of items a closed form (MaskedItems): tiles outside it are neither
//   read nor multiplied. 16,384 tokens in a window of 1,024: 265 us (all of them: 1,393).
// - A cap is a polynomial (shape_scores): five multiply-adds a column more, which is what bounds it
//   (tensor cores 47 % busy at 4,096 tokens): 16,384 tokens capped at 50: 1.61 ms, 1.36 PFLOP/s, 72 % of
//   cuBLAS's burst. Capped scores lie in a known range, so a row keeps the reference that its first keys
//   give (no maximum, no rescaling).
// - A bias grows towards the row's own position: key tiles are taken from the last one back, so that the
//   reference is found in the first. 24 prompts of 33 to 2,500 tokens: 364 us, 51 %.
// - The code of a tile decides as much as its operations: the instruction cache is shared by eight softmax
//   warps that are never at the same place. So there is one short path for tiles that all rows see (fast_tile,
//   fast_parts) and one for all others, in a loop of 32 columns. Masks in the fast path cost more than they
//   saved (64 prompts of 300 tokens capped: 153 -> 217 us), and so did shaping an item's first tile twice for its
//   reference (153 -> 170; a pass over its raw products instead, see begin_fixed: 148 -> 146).
// 64 decodes in a window of 4,096 keys, capped, pages of 16: 169 us, 5.7 TB/s, 84 % (without options over
// as many keys 180).
//
// 12 warps: two softmax warpgroups (thread = row: a tcgen05.ld gives a thread
// its whole row of S, no shuffles), one warp that issues the MMAs, one that loads K
// and V by TMA (128-byte swizzle; a ring of tiles), one that loads Q and sends staged
// rows off, and one that hands out the items (its code would cost every other role the
// instruction cache). Waits are bounded: one that gives up flags HA_DEVERR_TIMEOUT, stops
// the other roles, lets the copies and products in flight land and frees the tensor
// memory before the CTA exits.
#pragma once

#include <climits>
#include <type_traits>

#include "packed_order.h"
#include "tc_common.cuh"

namespace ha {
namespace {

constexpr int kAttThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kQWarp = 10, kPlanWarp = 11;
// Registers of a softmax thread and of the others: 256 x 216 + 128 x 72 is what 384
// threads are launched with (168 each).
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr int kMinSpan = 2;           // least work of a CTA (a token over 700 keys, 2 KV heads: 14.8 us; with 3: 16.1)
constexpr uint32_t kTmemCols = 512;   // S0, S1 (128 each; P overlays them), O0, O1
// Tiles that an item's start and end cost beside its own (24 prompts 331 us; 1: 343, 4: 354),
// and that writing a part of an item and joining it cost (64 prompts of up to 500 tokens
// 150 us, 1: 157; 64 decodes 338 us, 8: 343).
constexpr int kItemCost = 2, kSplitCost = 4;
constexpr int kQueue = 4;              // segments that the scheduler is ahead
constexpr float kRescale = 8.f;       // growth of the maximum (log2) that makes O be rescaled
// The same for shaped scores, where it sends a tile's rest the slow way: weights up to 2^40 cost no more
// range or precision than up to 2^8.
constexpr float kShapedRescale = 40.f;

// FOLD: the halves of a K/V tile lie side by side (PackedParams::kv_fold != 0)
template <int D, bool F32OUT, bool FOLD>
struct AttCfg {
    static constexpr int kKeys = F32OUT ? 64 : 128;      // keys per tile
    static constexpr int kHalves = D / 64;               // 128-byte swizzle spans of a row
    static constexpr int kQTile = 128 * D * 2;           // bytes of a Q tile
    static constexpr int kTile = kKeys * D * 2;          // bytes of a K or V tile
    // its 8-row groups of one half lie kGroup bytes apart, its halves kSpan
    static constexpr int kGroup = FOLD ? 2048 : 1024, kSpan = FOLD ? 1024 : kKeys * 128;
    static constexpr int kStages = 5 * 32768 / kTile;
    static constexpr int kParts = F32OUT ? 3 : 1;        // bf16 parts of P
    // First tensor memory column of a part: P takes the columns of S; three parts of 32
    // columns take the second half, beside S's 64, and S's first 32 once they are read.
    static constexpr __host__ __device__ int part_col(int i) { return !F32OUT || i == 2 ? 0 : 64 + 32 * i; }
    // Places for S and P: one to a stream where O leaves no more room; else three that the
    // products take in turn, so that S runs up to three products ahead of P V.
    static constexpr int kPlaces = D == 64 ? 3 : 2;
    static constexpr int kOCols = D == 64 ? 64 : 128;
    static constexpr __host__ __device__ uint32_t place_col(uint32_t b) { return b < 2u ? b * 128u : 384u; }
    // Whole rows of bf16 output leave by TMA (see `staged` below): 24 prompts 338 -> 331 us, 64 of
    // up to 500 tokens 152 -> 141. At d 64 there is half as much to write, and it cost (16,384
    // tokens 1106 -> 1151).
    static constexpr bool kStaged = !F32OUT && D == 128;
    static_assert(!kStaged || kStages <= 5, "a staged item's second slot waits for the staged item before");
    static constexpr int kBars = (2 * kStages + 8 + 3 * kPlaces + 2 * kQueue + 1) & ~1;  // the segments behind them are read as vectors
    static constexpr int kSmem = 2 * kQTile + kStages * kTile + 2048 + 8 * kBars + 64 * kQueue + 16 + kKeys;
    static_assert(kSmem <= 232448, "shared memory of a CTA");
};

struct SeqInfo {
    int q0, nq, nk;
};
// With score options: the first key that the sequence sees, and the end of the keys that all its
// tokens see (both within [0, nk]).
struct SeqInfoEx : SeqInfo {
    int first, prefix;
};
template <bool EX>
using Info = std::conditional_t<EX, SeqInfoEx, SeqInfo>;
template <bool EX>
using Params = std::conditional_t<EX, PackedParamsEx, PackedParams>;

// Sequence s, or an empty one (flagged) where its bounds are bad.
template <bool EX>
__device__ __forceinline__ Info<EX> seq_info(const Params<EX>& p, int s, bool report) {
    Info<EX> i;
    const int a = p.cu[s], b = p.cu[s + 1];
    const bool bad = a < 0 || b < a || b > p.total;
    i.q0 = a;
    i.nq = bad ? 0 : b - a;
    i.nk = i.nq;
    bool badk = false;
    if (p.seq_lens != nullptr) {
        i.nk = p.seq_lens[s];
        badk = i.nk < 0 || i.nk > p.max_len;
        if (badk) i.nk = 0;
    }
    if (report && (bad || badk)) flag_error(p.err, HA_DEVERR_SEQLEN);
    if constexpr (EX) {
        i.first = p.first != nullptr ? min(max(p.first[s], 0), i.nk) : 0;
        i.prefix = p.prefix != nullptr ? min(max(p.prefix[s], 0), i.nk) : 0;
    }
    return i;
}
// Lane `at`'s sequence.
template <bool EX>
__device__ __forceinline__ Info<EX> seq_of(const Info<EX>& i, int at) {
    Info<EX> r;
    r.q0 = __shfl_sync(0xffffffffu, i.q0, at);
    r.nq = __shfl_sync(0xffffffffu, i.nq, at);
    r.nk = __shfl_sync(0xffffffffu, i.nk, at);
    if constexpr (EX) {
        r.first = __shfl_sync(0xffffffffu, i.first, at);
        r.prefix = __shfl_sync(0xffffffffu, i.prefix, at);
    }
    return r;
}

// End of the keys that the first `upto` new tokens of the sequence see.
__device__ __forceinline__ int keys_seen(const SeqInfo& i, int upto) {
    const int k = i.nk - i.nq + min(upto, i.nq);
    return max(k, 0);
}
__device__ __forceinline__ int keys_seen(const SeqInfoEx& i, int upto) {
    return max(i.nk - i.nq + min(upto, i.nq), i.prefix);
}

template <int KT>
__device__ __forceinline__ int key_tiles(int keys) {
    return (keys + KT - 1) / KT;
}

// Cost of the items 0 .. qt - 1 of one head, qt < the number of items: their tiles
// (an item without keys counts one, so that its rows are written) and kItemCost each.
struct Window {  // what the work of an item takes from the options, beside its sequence
    int keys;
    Quotient per;
};

template <int KT>
struct Tiles {
    static constexpr int kLog = KT == 64 ? 6 : 7;
    TileSums<kLog> sums;
    const uint16_t* before;  // (shared memory)
};

template <int KT>
__device__ __forceinline__ uint32_t cost_before(const SeqInfo& i, const Window&, int t2, int qt, const Tiles<KT>& tiles) {
    if (qt == 0) return 0;
    const int base = i.nk - i.nq;
    int z = 0;  // items that see no key
    if (base < 0) z = min(qt, (-base) / t2);
    uint32_t c = (uint32_t)z + (uint32_t)qt * kItemCost;
    if (qt > z) c += tiles.sums.sum((uint32_t)(qt - z), (uint32_t)(base + (z + 1) * t2 + KT - 1), tiles.before);
    return c;
}

template <int KT>
__device__ __forceinline__ int item_tiles(const SeqInfo& i, const Window&, int t2, int qt) {
    return max(1, key_tiles<KT>(keys_seen(i, (qt + 1) * t2)));
}

// With score options.
template <int KT>
__device__ __forceinline__ MaskedItems<Tiles<KT>::kLog> masked(const SeqInfoEx& i, const Window& window, int t2) {
    return MaskedItems<Tiles<KT>::kLog>{i.nk - i.nq, i.nq, i.first, i.prefix, window.keys, t2, window.per};
}
template <int KT>
__device__ __forceinline__ uint32_t cost_before(const SeqInfoEx& i, const Window& window, int t2, int qt, const Tiles<KT>& tiles) {
    return masked<KT>(i, window, t2).tiles_before(qt, tiles.sums, tiles.before) + (uint32_t)qt * kItemCost;
}
template <int KT>
__device__ __forceinline__ int item_tiles(const SeqInfoEx& i, const Window& window, int t2, int qt) {
    return masked<KT>(i, window, t2).tiles(qt);
}

template <int KT, typename I>
__device__ __forceinline__ uint32_t head_cost(const I& i, const Window& window, int t2, const Tiles<KT>& tiles) {
    if (i.nq == 0) return 0;
    const int last = (i.nq + t2 - 1) / t2 - 1;
    return cost_before<KT>(i, window, t2, last, tiles) + (unsigned)(item_tiles<KT>(i, window, t2, last) + kItemCost);
}

// A place in the order of all work: tile j of item (s, head, qt), after w units.
struct Place {
    uint32_t w;
    int s, head, qt, j;
};

// The part of an item that this CTA works on, as the scheduler warp hands it to the
// others (16 ints in shared memory).
struct alignas(16) Segment {
    int nt;       // its key tiles (0: an item without keys; -1: no more)
    int jb;       // the first of them
    int e0;       // two row tiles: those that row tile 0 sees; else nt
    int flags;    // 1: one row tile (streams take every other key tile); 2: the whole item;
                  // 4: its rows four times, once for each warp of a stream
    int row0;     // row of its first token in q, out, lse
    int head;     // KV head
    int kend;     // keys that its last token sees
    int tokens;
    int kfirst;   // keys that the token before its first one sees (below 0: none, by that many)
    int nk;       // keys of the sequence
    int s, q0;    // sequence and its first row
    int begins;   // the item begins here
    // with score options
    int prefix;   // keys below it are seen by every token (but those below a row's first)
    int first;    // the sequence's first key
    int kbegin;   // the first key that the item's first token sees
};

template <int T>
struct Stream {
    static constexpr int value = T;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two float32 lanes of a 64-bit register.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// two bf16 values, the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// x[k] for a row that sees the first lim of n columns: -inf from there on.
template <int N>
__device__ __forceinline__ void mask_columns(uint32_t (&x)[N], int lim) {
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k >= lim) x[k] = 0xff800000u;
}

// max(a, max of x): four chains, so that they overlap.
template <int N>
__device__ __forceinline__ float max_of(const uint32_t (&x)[N], float a) {
    float m[4] = {a, a, a, a};
#pragma unroll
    for (int k = 0; k < N; k += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u)
            m[u] = fmaxf(fmaxf(m[u], __uint_as_float(x[k + 2 * u])), __uint_as_float(x[k + 2 * u + 1]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// The weights 2^{x qscale - sub} of 32 columns as bf16 pairs in w; their float32 sum is
// added to sum, and mt takes part in the columns' maximum.
// PLAIN: the weights 2^x.
template <bool PLAIN = false>
__device__ __forceinline__ void weights32(const uint32_t* x, uint64_t qscale2, uint64_t nsub2, uint32_t (&w)[16],
                                          uint64_t (&sum)[2]) {
#pragma unroll
    for (int q = 0; q < 16; q += 4) {
        float e[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (PLAIN) {
                e[2 * k] = __uint_as_float(x[2 * (q + k)]);
                e[2 * k + 1] = __uint_as_float(x[2 * (q + k) + 1]);
            } else {
                unpack2(fma2(pack2(__uint_as_float(x[2 * (q + k)]), __uint_as_float(x[2 * (q + k) + 1])), qscale2, nsub2), e[2 * k], e[2 * k + 1]);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = ex2(e[k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            w[q + k] = pack_bf16(e[2 * k], e[2 * k + 1]);
            sum[k & 1] = add2(sum[k & 1], pack2(e[2 * k], e[2 * k + 1]));
        }
    }
}

// Output rows of a pair of lanes (the even one's and the odd one's; null: not written).
// A lane holds a row, so its stores of 16 or 32 bytes would touch 32 rows at a time and
// cost as many tag lookups (5,700 cycles for two row tiles). The lanes of a pair swap
// halves and write one row together: 16 rows at a time, twice the bytes each (24 ragged
// prompts: 440 -> 371 us), in stores of 32 bytes where `out` starts on such a boundary
// (338 us; in stores of 16: 362).
struct RowPair {
    char *even, *odd;
    bool is_odd;
};
__device__ __forceinline__ RowPair pair_rows(char* mine, bool valid, int lane) {
    const unsigned long long m = valid ? (unsigned long long)mine : 0ull;
    const unsigned long long o = __shfl_xor_sync(0xffffffffu, m, 1);
    RowPair r;
    r.is_odd = (lane & 1) != 0;
    r.even = reinterpret_cast<char*>(r.is_odd ? o : m);
    r.odd = reinterpret_cast<char*>(r.is_odd ? m : o);
    return r;
}

__device__ __forceinline__ void store32(char* dst, const uint32_t* w, bool aligned32) {
    if (aligned32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// N words of this lane's row, `off` bytes into it.
template <int N>
__device__ __forceinline__ void store_rows(const uint32_t (&w)[N], const RowPair& r, int off, bool aligned32) {
    uint32_t keep[N / 2], got[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        keep[k] = r.is_odd ? w[N / 2 + k] : w[k];
        got[k] = __shfl_xor_sync(0xffffffffu, r.is_odd ? w[k] : w[N / 2 + k], 1);
    }
    off += r.is_odd ? N * 2 : 0;
    uint32_t e[N / 2], o[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
        e[k] = r.is_odd ? got[k] : keep[k];
        o[k] = r.is_odd ? keep[k] : got[k];
    }
#pragma unroll
    for (int k = 0; k < N / 2; k += 8) {
        if (r.even != nullptr) store32(r.even + off + 4 * k, e + k, aligned32);
        if (r.odd != nullptr) store32(r.odd + off + 4 * k, o + k, aligned32);
    }
}

// The weights 2^{x qscale - sub} of 16 columns as three bf16 parts each (pairs in q); returns
// their float32 sum.
// PLAIN: of the weights 2^x.
template <int N, bool PLAIN = false>
__device__ __forceinline__ float parts16(const uint32_t (&x)[N], float qscale, float sub, uint32_t (&q)[3][8]) {
    static_assert(N == 16, "three parts of 16 columns");
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float u = ex2(PLAIN ? __uint_as_float(x[2 * k]) : fmaf(__uint_as_float(x[2 * k]), qscale, -sub));
        float v = ex2(PLAIN ? __uint_as_float(x[2 * k + 1]) : fmaf(__uint_as_float(x[2 * k + 1]), qscale, -sub));
        s0 += u;
        s1 += v;
#pragma unroll
        for (int e = 0; e < 3; ++e) {
            q[e][k] = pack_bf16(u, v);
            u -= bf16lo(q[e][k]);
            v -= bf16hi(q[e][k]);
        }
    }
    return s0 + s1;
}

// x[k] for a row that sees the columns from lo on: -inf before it.
template <int N>
__device__ __forceinline__ void mask_before(uint32_t (&x)[N], int lo) {
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (k < lo) x[k] = 0xff800000u;
}

// The bits of the columns lo <= k < hi, of 32.
__device__ __forceinline__ uint32_t column_bits(int lo, int hi) {
    const uint32_t below = hi >= 32 ? ~0u : (hi <= 0 ? 0u : (1u << hi) - 1u);
    return lo <= 0 ? below : (lo >= 32 ? 0u : below & (~0u << lo));
}
// -inf in the columns that are not seen.
template <int N>
__device__ __forceinline__ void mask_bits(uint32_t (&x)[N], uint32_t seen) {
#pragma unroll
    for (int k = 0; k < N; ++k)
        if ((seen >> k & 1u) == 0u) x[k] = 0xff800000u;
}

// Largest magnitude (NaN apart), and that of the columns that are seen.
template <int N>
__device__ __forceinline__ float magnitude(const uint32_t (&x)[N], uint32_t seen) {
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < N; ++k)
        if ((seen >> k & 1u) != 0u) m[k & 3] = fmaxf(m[k & 3], fabsf(__uint_as_float(x[k])));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
template <int N>
__device__ __forceinline__ float magnitude(const uint32_t (&x)[N]) {
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < N; k += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u)
            m[u] = fmaxf(fmaxf(m[u], fabsf(__uint_as_float(x[k + 2 * u]))), fabsf(__uint_as_float(x[k + 2 * u + 1])));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// x = f(x) of pairs of columns.
template <int N, typename F>
__device__ __forceinline__ void each_pair(uint32_t (&x)[N], F&& f) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        float a, b;
        unpack2(f(pack2(__uint_as_float(x[k]), __uint_as_float(x[k + 1]))), a, b);
        x[k] = __float_as_uint(a);
        x[k + 1] = __float_as_uint(b);
    }
}
// v (c[0] + c[1] v^2 + .. + c[DEG] v^{2 DEG}) + plus
template <int DEG>
__device__ __forceinline__ uint64_t odd_poly(uint64_t v, const float (&c)[7], uint64_t plus) {
    const uint64_t u = mul2(v, v);
    uint64_t y = pack2(c[DEG], c[DEG]);
#pragma unroll
    for (int i = DEG - 1; i >= 0; --i) y = fma2(y, u, pack2(c[i], c[i]));
    return fma2(v, y, plus);
}

// cap tanh(x scale / cap) log2(e), off by 2^-22 cap at most.
__device__ __forceinline__ float cap_of(float x, const PackedParamsEx& p) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(x * p.twice)));
    return fmaf(-2.f * p.cap, r, p.cap);
}

// Degrees of the polynomials for tanh(u) / u (PackedParamsEx::fit and poly).
template <bool F32OUT>
struct CapDegrees {
    static constexpr int low = F32OUT ? 4 : 3, high = F32OUT ? 6 : 5;
};

// Products x = <q, k_j> of consecutive columns as what the softmax takes the power of 2 of: the score
// (x scale, or capped cap tanh(x scale / cap)) less slope times the distance, times log2 e, less
// sub. `from`: the first column's key less the row's position (below 0: the key lies before it).
//
// The products of a float32 multiply and add are what a tile waits for (a pair of columns in one
// instruction takes as long as two), so tanh u is u P(u^2) with no more terms than the warp's
// largest |u| asks for, and no exponential or reciprocal: P is fitted in relative error, to
// 5.4e-7 at most (bf16 weights: they are rounded to 4e-3) or 5.0e-8 (float32 results: half a
// rounding). Beyond |u| = 1 it is 1 - 2 / (1 + e^{2 u}), off by 2^-22 cap at most. The choice shows in
// a result's last bits, so the largest product is that of tokens' rows, over the keys that they see
// (`mine`: this row's, 0 of a row of no token): whatever else lies in a tile of queries or keys has no part in it.
template <bool F32OUT, bool BIAS, int N>
__device__ __forceinline__ void shape_scores(uint32_t (&x)[N], const PackedParamsEx& p, float slope, float from, bool both_sides, float mine,
                                             float sub) {
    using Deg = CapDegrees<F32OUT>;
    const float row = BIAS && !both_sides ? fmaf(slope, from, -sub) : -sub;
    const uint64_t row2 = pack2(row, row);
    if (!BIAS || p.cap != 0.f) {
        const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mine)));
        if (top <= p.fit[0]) {
            each_pair(x, [&](uint64_t v) { return odd_poly<Deg::low>(v, p.poly[0], row2); });
        } else if (top <= p.fit[1]) {
            const uint64_t unit = pack2(p.unit, p.unit);
            each_pair(x, [&](uint64_t v) { return odd_poly<Deg::high>(mul2(v, unit), p.poly[1], row2); });
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = __float_as_uint(cap_of(__uint_as_float(x[k]), p) + row);
        }
    } else {
        const uint64_t s2 = pack2(p.scale, p.scale);
        each_pair(x, [&](uint64_t v) { return fma2(v, s2, row2); });
    }
    if (BIAS && p.slopes != nullptr) {
        if (!both_sides) {
#pragma unroll
            for (int k = 1; k < N; ++k) x[k] = __float_as_uint(fmaf(slope, (float)k, __uint_as_float(x[k])));
        } else {  // keys on both sides of the row's position
#pragma unroll
            for (int k = 0; k < N; ++k) x[k] = __float_as_uint(fmaf(-slope, fabsf(from + (float)k), __uint_as_float(x[k])));
        }
    }
}

__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&x)[16]) { tmem_ld16(addr, x); }
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&x)[32]) { tmem_ld32(addr, x); }

// Whether `x` holds in any of the warp's rows of tokens (valid, `tokens` by lane). LATE: all rows vote and the others
// are left out of the outcome (16,384 biased tokens at d 64: 1,241 us, with the condition in the vote 1,329; 24
// capped prompts of 1,000 with float32 results 359 and 366; 16,384 capped tokens with bf16 results 1,479 and 1,441).
template <bool LATE>
__device__ __forceinline__ bool of_tokens(bool x, bool valid, uint32_t tokens) {
    return LATE ? (__ballot_sync(0xffffffffu, x) & tokens) != 0u : (bool)__any_sync(0xffffffffu, valid && x);
}

// The weights of a tile of 128 columns of shaped scores, all seen, keys on one side of the rows: score k
// of the tile, less the reference, is x scale (CAP: the polynomial) + row, and with BIAS + slope k.
// Returns the columns done: those before the first 32 where a product of any of the warp's valid rows is too
// large for the polynomial, or (BIAS) a score more than kShapedRescale above the reference.
//
// 32 columns at a time in a loop: what bounds short prompts is the instruction cache, which the item's
// first and last tiles share with this code. UNROLL 4 lets the exponentials of 32 columns run under the
// multiplications of the next (in a kernel of its own: beside the loop it is no faster). Capped scores,
// loop / unrolled: 24 prompts of 1,000 tokens 261 / 303 us, 8 of 2,048 276 / 296, 4 of 4,096 469 / 480, one of
// 8,192 445 / 448, two of 8,192 857 / 851, one of 12,288 950 / 930, one of 16,384 1,640 / 1,605, one of 24,576
// 3,760 / 3,715; 64 decodes over up to 16,000 keys 343 / 348, in a window of 4,096 179 / 182, 48 over 500 to 1,500
// keys 56 / 62. At d 64 the loop was the faster at any length, and for biased ones at d 128 up to 4,096 tokens.
template <bool CAP, bool BIAS, int UNROLL>
__device__ __forceinline__ int fast_tile(uint32_t tS, const PackedParamsEx& p, float row, float slope, bool valid, uint64_t (&sum)[2]) {
    const uint64_t scale = pack2(p.scale, p.scale);
    const uint32_t tokens = __ballot_sync(0xffffffffu, valid);
#pragma unroll UNROLL
    for (int c0 = 0; c0 < 128; c0 += 32) {
        uint32_t x[32], w[16];
        uint64_t s[2] = {0, 0};
        float y[32], big[2] = {0.f, 0.f}, top[2] = {-INFINITY, -INFINITY};
        const float r = BIAS ? fmaf(slope, (float)c0, row) : row;
        const uint64_t row2 = pack2(r, r);
        tmem_ld32(tS + (uint32_t)c0, x);
        tmem_landed(x);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            const uint64_t v = pack2(__uint_as_float(x[k]), __uint_as_float(x[k + 1]));
            const int u = (k >> 1) & 1;
            if constexpr (CAP) {
                unpack2(odd_poly<CapDegrees<false>::low>(v, p.poly[0], row2), y[k], y[k + 1]);
                big[u] = fmaxf(fmaxf(big[u], fabsf(__uint_as_float(x[k]))), fabsf(__uint_as_float(x[k + 1])));
            } else {
                unpack2(fma2(v, scale, row2), y[k], y[k + 1]);
            }
            if constexpr (BIAS) {
                y[k] = fmaf(slope, (float)k, y[k]);
                y[k + 1] = fmaf(slope, (float)(k + 1), y[k + 1]);
                top[u] = fmaxf(fmaxf(top[u], y[k]), y[k + 1]);
            }
        }
        const bool stop = of_tokens<BIAS>((CAP && fmaxf(big[0], big[1]) > p.fit[0]) || (BIAS && fmaxf(top[0], top[1]) > kShapedRescale), valid, tokens);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
            const float a = ex2(y[k]), b = ex2(y[k + 1]);
            w[k >> 1] = pack_bf16(a, b);
            s[(k >> 1) & 1] = add2(s[(k >> 1) & 1], pack2(a, b));
        }
        if (stop) return c0;
        sum[0] = add2(sum[0], s[0]);
        sum[1] = add2(sum[1], s[1]);
        tmem_st16(tS + (uint32_t)(c0 >> 1), w);
    }
    return 128;
}

// The same for tiles of 64 columns and weights of three bf16 parts, 16 columns at a time.
template <bool CAP, bool BIAS>
__device__ __forceinline__ int fast_parts(uint32_t tS, const uint32_t (&part_at)[3], const PackedParamsEx& p, float row, float slope, bool valid,
                                          float& l) {
    const uint64_t scale = pack2(p.scale, p.scale);
    const uint32_t tokens = __ballot_sync(0xffffffffu, valid);
#pragma unroll 1
    for (int c0 = 0; c0 < 64; c0 += 16) {
        uint32_t x[16], q[3][8];
        float big = 0.f, top = -INFINITY;
        const float r = BIAS ? fmaf(slope, (float)c0, row) : row;
        const uint64_t row2 = pack2(r, r);
        tmem_ld16(tS + (uint32_t)c0, x);
        tmem_landed(x);
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
            float a = __uint_as_float(x[k]), b = __uint_as_float(x[k + 1]);
            const uint64_t v = pack2(a, b);
            if constexpr (CAP) {
                big = fmaxf(fmaxf(big, fabsf(a)), fabsf(b));
                unpack2(odd_poly<CapDegrees<true>::low>(v, p.poly[0], row2), a, b);
            } else {
                unpack2(fma2(v, scale, row2), a, b);
            }
            if constexpr (BIAS) {
                a = fmaf(slope, (float)k, a);
                b = fmaf(slope, (float)(k + 1), b);
                top = fmaxf(fmaxf(top, a), b);
            }
            x[k] = __float_as_uint(a);
            x[k + 1] = __float_as_uint(b);
        }
        const bool stop = of_tokens<true>((CAP && big > p.fit[0]) || (BIAS && top > kShapedRescale), valid, tokens);
        const float more = parts16<16, true>(x, 0.f, 0.f, q);
        if (stop) return c0;
        l += more;
#pragma unroll
        for (int e = 0; e < 3; ++e) tmem_st8(tS + part_at[e] + (uint32_t)(c0 >> 1), q[e]);
    }
    return 64;
}

// 2^x of the whole number nearest to x <= 0; 0 below what normal numbers reach.
__device__ __forceinline__ float whole_power(float x) {
    return x < -126.f ? 0.f : __int_as_float((127 + __float2int_rn(x)) << 23);
}

// a times the pairs of bf16 in 8 columns of tensor memory (a power of 2: exact).
__device__ __forceinline__ void scale_pairs8(uint32_t addr, float a) {
    uint32_t w[8];
    tmem_ld8(addr, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = pack_bf16(bf16lo(w[k]) * a, bf16hi(w[k]) * a);
    tmem_st8(addr, w);
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// What the softmax takes the scores as: they are scaled (kPlain: no options at all; kMasked: masks
// alone), capped with a reference that stays (kCapped; kCappedLong: of long items, see fast_tile), or
// shaped in any way (kShaped).
enum Mode { kPlain = 0, kMasked = 1, kCapped = 2, kCappedLong = 3, kShaped = 4 };

template <int D, bool F32OUT, bool FOLD, int MODE>
__global__ void __launch_bounds__(kAttThreads, 1)
    k_packed_att(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmQs,
                 const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const __grid_constant__ CUtensorMap tmO,
                 const Params<(MODE != kPlain)> p) {
    constexpr bool EX = MODE != kPlain, shaped = MODE >= kCapped, fixed = MODE == kCapped || MODE == kCappedLong;
    // Biased scores grow towards the row's own position, so key tiles are taken from the last one
    // back: the reference is found in the first, instead of moving (and O being rescaled) in most.
    constexpr bool BACK = MODE == kShaped;
    using C = AttCfg<D, F32OUT, FOLD>;
    constexpr int S = C::kStages, KT = C::kKeys, NB = C::kPlaces;
    extern __shared__ __align__(1024) uint8_t s_raw[];
    const uint32_t base = smem_addr(s_raw);
    const uint32_t s_q = base, s_ring = base + 2 * C::kQTile;
    uint8_t* g_tail = s_raw + 2 * C::kQTile + S * C::kTile;
    float2* s_ml = reinterpret_cast<float2*>(g_tail);                 // [2][128] (m, l) of the two warpgroups
    const uint32_t bars = base + (uint32_t)(2 * C::kQTile + S * C::kTile) + 2048u;
    uint8_t* g_misc = g_tail + 2048 + 8 * C::kBars;
    Segment* s_seg = reinterpret_cast<Segment*>(g_misc);              // [kQueue]
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(g_misc + kQueue * sizeof(Segment));
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    uint16_t* s_before = reinterpret_cast<uint16_t*>(s_tmem + 4);     // [kKeys / 2] (TileSums)
    auto full = [&](int s) { return bars + 8u * (uint32_t)s; };
    auto empty = [&](int s) { return bars + 8u * (uint32_t)(S + s); };
    auto bar_at = [&](int i) { return bars + 8u * (uint32_t)(2 * S + i); };
    const uint32_t q_full = bar_at(0), q_empty = bar_at(1), x_bar = bar_at(4 + 3 * NB), done = bar_at(5 + 3 * NB), seg_done = bar_at(6 + 3 * NB);
    // of a place (which is the stream's, where there are two); o_done: P V from it has finished
    auto s_full = [&](int b) { return bar_at(2 + b); };
    auto p_full = [&](int b) { return bar_at(2 + NB + b); };
    auto o_done = [&](int b) { return bar_at(2 + 2 * NB + b); };
    auto o_free = [&](int t) { return bar_at(2 + 3 * NB + t); };
    auto seg_full = [&](int i) { return bar_at(7 + 3 * NB + i); };
    const uint32_t staged_full = bar_at(7 + 3 * NB + 2 * kQueue);
    auto seg_read = [&](int i) { return bar_at(7 + 3 * NB + kQueue + i); };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((base & 1023u) != 0u) {  // the swizzle atoms need it; shared memory starts there
        pdl_wait();
        if (tid == 0) {
            p.items[blockIdx.x].parts = 0;
            flag_error(p.err, HA_DEVERR_STATE);
        }
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int b = 0; b < NB; ++b) {
            mbar_init(s_full(b), 1);
            mbar_init(p_full(b), 4);
            mbar_init(o_done(b), 1);
        }
        for (int t = 0; t < 2; ++t) mbar_init(o_free(t), 8);
        mbar_init(x_bar, 8);
        if (C::kStaged) mbar_init(staged_full, 8);
        mbar_init(done, 1);
        mbar_init(seg_done, 1);
        for (int i = 0; i < kQueue; ++i) {
            mbar_init(seg_full(i), 1);
            mbar_init(seg_read(i), kPlanWarp);  // every warp but the scheduler
        }
        *s_abort = 0;
        mbar_fence_init();
        tmap_prefetch(&tmQ);
        tmap_prefetch(&tmK);
        tmap_prefetch(&tmV);
    }
    if (warp == kMmaWarp) tmem_alloc(smem_addr(s_tmem), kTmemCols);
    const int t2 = 2 * p.TQ;
    Window window{};
    if constexpr (EX) window = Window{p.window, p.per_item};
    const Tiles<KT> tiles{TileSums<Tiles<KT>::kLog>((uint32_t)t2), s_before};
    if (warp == kPlanWarp) {
        // sums of remainders, two a lane at most
        constexpr int per = KT / 64;
        uint32_t r[per], incl = 0;
#pragma unroll
        for (int u = 0; u < per; ++u) incl += r[u] = tiles.sums.remainder((uint32_t)(per * lane + u));
        uint32_t at = incl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        at = incl - at;
#pragma unroll
        for (int u = 0; u < per; ++u) {
            s_before[per * lane + u] = (uint16_t)at;
            at += r[u];
        }
        __syncwarp();
    }
    pdl_wait();
    pdl_launch_dependents();  // behind the wait, so that what the next kernel may find running is this one alone

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    auto give_up = [&]() {
        flag_error(p.err, HA_DEVERR_TIMEOUT);
        *s_abort = 1;
    };
    auto wait = [&](uint32_t bar, uint32_t parity) {
        mbar_wait_or_abort(bar, parity, s_abort);
        tc_fence_after();
    };
    auto aborted = [&]() { return (bool)__any_sync(0xffffffffu, *s_abort != 0); };
    // The next segment (n counts them): false when there is none, or after a timeout.
    auto next_segment = [&](int& n, Segment& g) {
        const int i = n % kQueue;
        wait(seg_full(i), (uint32_t)(n / kQueue) & 1u);
        g = s_seg[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(seg_read(i));
        ++n;
        return !aborted() && g.nt >= 0;
    };
    // bf16 rows of a whole item of two row tiles leave through the ring: behind the item's
    // tiles come two slots that the loader passes by. A softmax warpgroup puts its rows
    // there, the Q warp sends them off by TMA (rows as Q's) and frees the slots. A row tile that
    // is not full is written row by row, as its box would reach past the sequence.
    auto staged = [&](const Segment& x) { return C::kStaged && (x.flags & 3) == 2 && x.nt > 0; };
    Segment g;
    int nseg = 0;

    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == kPlanWarp) {
            // ---- this CTA's range of work, then its items in order
            // Sequences are taken 32 at a time, one to a lane; a batch stays in registers (the first,
            // until the items are handed out).
            Info<EX> batch{}, i{};
            auto load = [&](int s, bool report) { return s < p.n_seq ? seq_info<EX>(p, s, report) : Info<EX>{}; };
            auto cost = [&](const Info<EX>& i) { return (uint32_t)p.Hkv * head_cost<KT>(i, window, t2, tiles); };
            int batch0 = 0;  // the batch's first sequence
            auto info_of = [&](int s) {
                if (s >= batch0 + 32) {
                    batch0 = s;
                    batch = load(s + lane, false);
                }
                return seq_of<EX>(batch, s - batch0);
            };
            uint32_t U = 0, cost0 = 0;
            int rows = 0;  // of this lane's sequences, as far as it matters
#pragma unroll 1
            for (int s0 = 0; s0 < p.n_seq; s0 += 32) {
                i = load(s0 + lane, blockIdx.x == 0);
                const uint32_t c = cost(i);
                if (s0 == 0) {
                    batch = i;
                    cost0 = c;
                }
                U += c;
                rows = min(rows + i.nq, 1 << 25);
            }
            U = __reduce_add_sync(0xffffffffu, U);
            // Bounds that go back (flagged above) can make the others overlap. Their work may
            // not be what the host has bounded, so nothing is done then.
            if (__reduce_add_sync(0xffffffffu, rows) > p.total) U = 0;
            // CTAs that work: as many as there are spans of kMinSpan
            const uint32_t P = min(max(U / kMinSpan, 1u), gridDim.x);
            const uint32_t span = U / P, over = U - span * P;  // boundary c: c U / P
            auto boundary = [&](uint32_t c) { return span * c + over * c / P; };
            // a boundary close to an item's edge moves to it: within an eighth of a span, and
            // within what parting the item would cost (always, where items are not parted)
            const uint32_t tol = p.split ? min(span / 8, (uint32_t)kSplitCost) : U;
            if (lane == 0) p.items[blockIdx.x].parts = 0;
            // The places of this CTA's two boundaries at once, one to each half of the warp.
            const int half = lane >> 4;
            const uint32_t c = blockIdx.x + (uint32_t)half;
            const bool inside = c < P && U != 0;
            const uint32_t bnd = inside ? boundary(c) : U, b0 = __shfl_sync(0xffffffffu, bnd, 0), b1 = __shfl_sync(0xffffffffu, bnd, 16);
            Place a{U, 0, 0, 0, 0};
            Info<EX> ai{};
            uint32_t rem = 0, whole_seq = 1;
            {
                bool open = inside;
                uint32_t before = 0;
#pragma unroll 1
                for (int s0 = 0; __any_sync(0xffffffffu, open); s0 += 32) {
                    if (s0 > 0) i = load(s0 + lane, false);
                    else i = batch;
                    const uint32_t mine = s0 == 0 ? cost0 : cost(i);
                    uint32_t incl = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o) incl += v;
                    }
                    const uint32_t m0 = __ballot_sync(0xffffffffu, b0 < before + incl), m1 = __ballot_sync(0xffffffffu, b1 < before + incl);
                    const uint32_t m = half ? m1 : m0;
                    const int at = m != 0 ? __ffs((int)m) - 1 : 31;
                    const uint32_t end = __shfl_sync(0xffffffffu, incl, at), own = __shfl_sync(0xffffffffu, mine, at);
                    const Info<EX> ii = seq_of<EX>(i, at);
                    if (open && m != 0) {
                        open = false;
                        a.s = s0 + at;
                        a.w = bnd;
                        ai = ii;
                        rem = bnd - before - (end - own);
                        whole_seq = own;
                    }
                    before += __shfl_sync(0xffffffffu, incl, 31);
                }
            }
            {
                const uint32_t uh = whole_seq / (uint32_t)p.Hkv;
                if (inside) a.head = (int)(rem / uh);
                rem -= uh * (uint32_t)a.head;
                // the last item that begins at or before rem, 16 of them a step
                int lo = 0, n = inside ? (ai.nq + t2 - 1) / t2 : 1;
                uint32_t begins = 0;
#pragma unroll 1
                while (__any_sync(0xffffffffu, n > 1)) {
                    const int step = (n + 15) >> 4, q = (lane & 15) * step;
                    const uint32_t at = q < n ? cost_before<KT>(ai, window, t2, lo + q, tiles) : ~0u;
                    const uint32_t m = __ballot_sync(0xffffffffu, at <= rem) >> (16 * half) & 0xffffu;
                    const int k = 31 - __clz((int)(m | 1u));
                    begins = __shfl_sync(0xffffffffu, at, 16 * half + k);
                    lo += k * step;
                    n = min(step, n - k * step);
                }
                const uint32_t off = rem - begins;
                const int len = item_tiles<KT>(ai, window, t2, lo);
                const uint32_t to_end = (uint32_t)(len + kItemCost) - off;
                a.qt = lo;
                a.j = max((int)off - kItemCost, 0);
                if (inside) {
                    if (off <= kItemCost || (off <= tol && off <= to_end)) {
                        a.w -= off;
                        a.j = 0;
                    } else if (to_end <= tol) {
                        a.w += to_end;
                        a.j = len;
                    }
                }
            }
            const uint32_t w0 = __shfl_sync(0xffffffffu, a.w, 0), w1 = __shfl_sync(0xffffffffu, a.w, 16);
            uint32_t left = w1 - w0;
            int s = __shfl_sync(0xffffffffu, a.s, 0), head = __shfl_sync(0xffffffffu, a.head, 0);
            int qt = __shfl_sync(0xffffffffu, a.qt, 0), j = __shfl_sync(0xffffffffu, a.j, 0), n = 0;
            i = seq_of<EX>(ai, 0);
            int nqt = (i.nq + t2 - 1) / t2;
            // The rest of an item that began in the CTA before comes last: all CTAs begin at a first
            // key, so those with items of the same K and V read them together (4 x 512 tokens over
            // 20,000 to 32,000 keys: 594 -> 574 us, under the power cap 672 -> 631).
            Segment held;
            held.nt = -1;
            bool more = left > 0, stop = false;
#pragma unroll 1
            while (!stop) {
                Segment o{};
                o.nt = -1;
                bool goes_on = false;  // the item begins here and goes on in the next CTAs
                uint32_t rest_after = 0;
                if (more) {
                    const int len = item_tiles<KT>(i, window, t2, qt);
                    if (j < len) {
                        const uint32_t rest = (uint32_t)(len - j + (j == 0 ? kItemCost : 0));
                        const int je = rest <= left ? len : j + (int)left - (j == 0 ? kItemCost : 0);
                        left -= rest <= left ? rest : left;
                        o.jb = j;
                        o.kend = keys_seen(i, (qt + 1) * t2);
                        int begin = 0;
                        bool none = false;
                        if constexpr (EX) {
                            o.prefix = i.prefix;
                            o.first = i.first;
                            const auto items = masked<KT>(i, window, t2);
                            o.kbegin = items.begin(qt * t2);
                            none = items.none(qt);
                            begin = items.begin_tile(qt);
                            o.jb += begin;
                        }
                        o.nt = none ? 0 : max(0, min(je, key_tiles<KT>(o.kend) - begin) - j);
                        o.tokens = min(t2, i.nq - qt * t2);
                        const bool one = o.tokens <= p.TQ;
                        // (from the last tile back, row tile 0 takes all, too: the ones that it sees come last)
                        o.e0 = one || none || BACK ? o.nt : max(0, min(je, key_tiles<KT>(keys_seen(i, qt * t2 + p.TQ)) - begin) - j);
                        // (spread: a token over 131,072 keys 118 us, without 137; whole items have
                        // other warps' rows to fill the time, and no merge to add up the quarters)
                        const bool whole = j == 0 && je == len, spread = !whole && o.tokens <= p.TS;
                        o.flags = (one ? 1 : 0) | (whole ? 2 : 0) | (spread ? 4 : 0);
                        o.row0 = i.q0 + qt * t2;
                        o.head = head;
                        o.kfirst = i.nk - i.nq + qt * t2;
                        o.nk = i.nk;
                        o.s = s;
                        o.q0 = i.q0;
                        o.begins = j == 0;
                        goes_on = j == 0 && je < len;
                        rest_after = (uint32_t)(len - je);
                    }
                    // the next item
                    j = 0;
                    if (++qt >= nqt) {
                        qt = 0;
                        if (++head >= p.Hkv) {
                            head = 0;
                            if (left > 0) {
                                ++s;
                                if (s < p.n_seq) i = info_of(s);
                                // Sequences without new tokens are passed by 32 at a time: one at a time (two
                                // dependent loads each) a few hundred thousand outlast the others' waits.
#pragma unroll 1
                                while (s < p.n_seq && i.nq == 0) {
                                    const uint32_t some = __ballot_sync(0xffffffffu, load(s + 1 + lane, false).nq > 0);
                                    s += some != 0 ? __ffs((int)some) : 32;
                                    if (some != 0) i = info_of(s);
                                }
                                if (s >= p.n_seq) left = 0;
                                nqt = (i.nq + t2 - 1) / t2;
                            }
                        }
                    }
                    more = left > 0;
                    if (o.nt < 0 && more) continue;  // the first place was an item's end
                    if ((EX ? o.begins == 0 : o.jb > 0) && more) {
                        held = o;
                        continue;
                    }
                } else if (held.nt >= 0) {
                    o = held;
                    held.nt = -1;
                }
                wait(seg_read(n % kQueue), ((uint32_t)(n / kQueue) & 1u) ^ 1u);
                if (lane == 0) {
                    s_seg[n % kQueue] = o;
                    mbar_arrive(seg_full(n % kQueue));
                }
                __syncwarp();
                if (goes_on && lane == 0) {
                    // what the merge needs: it ends at the first boundary that has reached it (within tol)
                    const uint32_t last = w1 + rest_after - tol;
                    uint32_t end = min((uint32_t)((float)last / (float)U * (float)P), P);  // off by one at most
                    while (end > 0 && (end == P ? U : boundary(end)) >= last) --end;
                    while (end < P && boundary(end) < last) ++end;
                    SplitItem d;
                    d.parts = (int)(end - blockIdx.x);
                    d.row0 = o.row0;
                    d.head = o.head;
                    d.tokens = (o.flags & 4) != 0 ? -o.tokens : o.tokens;
                    p.items[blockIdx.x] = d;
                }
                __syncwarp();
                ++n;
                stop = o.nt < 0 || aborted();
            }
        } else if (warp == kQWarp) {
            int nq = 0;
            uint32_t ring = 0, sent = 0, slot = 0;  // ring tiles, staged items so far; the pending one's slot
            int row0 = -1, head = 0, tiles = 0;     // the pending item: its first row (-1: none), full row tiles
            auto send = [&]() {
                if (!C::kStaged || row0 < 0) return;
                wait(staged_full, sent & 1u);
                ++sent;
                if (lane == 0) {
                    if (*s_abort == 0) {
                        for (int t = 0; t < tiles; ++t)
                            for (int h = 0; h < C::kHalves; ++h)
                                tma_store_4d(&tmO, s_ring + (slot + (uint32_t)t) % (uint32_t)S * (uint32_t)C::kTile + (uint32_t)(h * 16384),
                                             h * 64, 0, row0 + t * p.TQ, head);
                        tma_store_read();
                    }
                    for (int t = 0; t < 2; ++t) mbar_arrive(empty((int)((slot + (uint32_t)t) % (uint32_t)S)));
                }
                __syncwarp();
                row0 = -1;
            };
#pragma unroll 1
            while (next_segment(nseg, g)) {
                if (g.nt == 0) continue;
                wait(q_empty, (uint32_t)(nq & 1) ^ 1u);
                if (aborted()) break;
                const bool spread = (g.flags & 4) != 0;
                const int copies = spread ? 4 : ((g.flags & 1) ? 1 : 2);
                if (lane == 0) mbar_arrive_expect_tx(q_full, (uint32_t)(copies * (spread ? p.TS : p.TQ) * p.G * D * 2));
                __syncwarp();
                if (lane < copies * C::kHalves) {
                    const int t = lane / C::kHalves, h = lane % C::kHalves;
                    tma_load_4d(s_q + (uint32_t)((spread ? t * 4096 : t * C::kQTile) + h * 16384), spread ? &tmQs : &tmQ, q_full,
                                h * 64, 0, g.row0 + (spread ? 0 : t * p.TQ), g.head);
                }
                ++nq;
                send();
                if (C::kStaged) ring += 2u * (uint32_t)g.nt;
                if (staged(g)) {
                    row0 = g.row0;
                    head = g.head;
                    tiles = g.tokens == t2 ? 2 : 1;
                    slot = ring;
                    ring += 2u;
                }
            }
            send();
            if (C::kStaged && lane == 0) tma_store_done();
            __syncwarp();
            // before the CTA can exit: the products have read it, or at least it has landed
            if (lane == 0 && nq > 0) mbar_wait_drain(*s_abort == 0 ? q_empty : q_full, (uint32_t)(nq - 1) & 1u);
        } else if (warp == kLoadWarp) {
            const int lg = p.box_log2;               // rows of a copy: 2^lg
            const int nbox = KT >> lg;
            // a copy takes one 64-dim half of its rows, or (pages, d = 128) both
            const int box = lane & (nbox - 1), half = lane / nbox, halves = FOLD ? 1 : C::kHalves;
            const uint32_t box_at = FOLD ? (uint32_t)(box << lg) * 256u : (uint32_t)(half * C::kSpan + (box << lg) * 128);
            int n = 0;
            bool ok = true;
#pragma unroll 1
            while (ok && next_segment(nseg, g)) {
                if (g.nt == 0) continue;
                const int jend = g.jb + g.nt;
                const int32_t* table = p.table != nullptr ? p.table + (int64_t)g.s * p.table_st : nullptr;
                // Page and row of this lane's box of tile j. The entry is looked at when the tile's
                // turn comes, so that its load does not hold up the tile before.
                auto where = [&](int j, int& page, int& row) {
                    const int key = j * KT + (box << lg);
                    page = 0;
                    row = g.q0 + key;
                    if (table != nullptr && key < g.kend) {
                        const int e = key / p.page_size;
                        row = key - e * p.page_size;
                        page = table[e];
                    }
                };
                int page_n, row_n;
                where(BACK ? jend - 1 : g.jb, page_n, row_n);
#pragma unroll 1
                for (int i = g.jb; ok && i < jend; ++i) {
                    const int j = BACK ? g.jb + jend - 1 - i : i;
                    const int boxes = (min(KT, g.kend - j * KT) + (1 << lg) - 1) >> lg;
                    // coordinates behind the dims: (row, head, page), or 8-row groups (see PackedParams)
                    int page = page_n, row = row_n;
                    if (i + 1 < jend) where(BACK ? j - 1 : j + 1, page_n, row_n);
                    // what lies before the item's first key may have been given away: its entries say nothing
                    const bool gone = EX && j == g.jb && j * KT + ((box + 1) << lg) <= g.kbegin;
                    if (table != nullptr && (page < 0 || page >= p.n_pages || gone)) {
                        if (!gone) flag_error(p.err, HA_DEVERR_INDEX);
                        page = p.n_pages;  // past the pool: the copy fills its rows with zeros
                        row = 0;
                    }
                    int c1 = row, c2 = g.head, c3 = page;
                    if (FOLD) {
                        c1 = (p.kv_fold == 1 ? page * p.page_size + row : row) >> 3;
                        if (p.kv_fold == 2) c2 = page < p.n_pages ? page * p.Hkv + g.head : p.n_pages * p.Hkv;
                    }
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv) {
                        const int s = n % S;
                        wait(empty(s), ((uint32_t)(n / S) & 1u) ^ 1u);
                        if (aborted()) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(full(s), (uint32_t)((boxes << lg) * D * 2));
                        __syncwarp();
                        if (box < boxes && half < halves) {
                            const CUtensorMap* tm = kv == 0 ? &tmK : &tmV;
                            const uint32_t dst = s_ring + (uint32_t)(s * C::kTile) + box_at;
                            if (FOLD) tma_load_5d(dst, tm, full(s), 0, 0, 0, c1, c2);
                            else tma_load_4d(dst, tm, full(s), half * 64, c1, c2, c3);
                        }
                        ++n;
                    }
                }
                if (ok && staged(g)) {
#pragma unroll 1
                    for (int t = 0; t < 2; ++t, ++n) {
                        wait(empty(n % S), ((uint32_t)(n / S) & 1u) ^ 1u);
                        if (lane == 0) mbar_arrive(full(n % S));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) {
                // before the CTA can exit: the products have released the last stages, or,
                // after a timeout, at least the copies into them have landed
                const bool clean = *s_abort == 0;
                for (int j = (n > S ? n - S : 0); j < n; ++j)
                    mbar_wait_drain(clean ? empty(j % S) : full(j % S), (uint32_t)(j / S) & 1u);
            }
        } else {
            constexpr uint32_t kIdS = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(KT >> 3) << 17) | ((128u >> 4) << 24);
            constexpr uint32_t kIdO = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(D >> 3) << 17) |
                                      ((128u >> 4) << 24);
            int nq = 0;
            uint32_t cnt = 0;  // bit t: parity of stream t's tiles so far
            uint32_t sb = 0, pb = 0, pph = 0;  // three places: that of the next S and P, and P's phase
            // Descriptors: Q (K-major, leading offset unused), the first ring slot as K (the same)
            // and as V, whose keys are the MMA's K dimension and the rows of the layout (MN-major).
            constexpr uint32_t kv_hi = sw128_desc_hi(C::kGroup);
            const uint32_t q_lo = uniform(((s_q & 0x3FFFFu) >> 4) | (1u << 16));
            const uint32_t k_lo = uniform(((s_ring & 0x3FFFFu) >> 4) | (1u << 16));
            const uint32_t v_lo = uniform(((s_ring & 0x3FFFFu) >> 4) | ((uint32_t)(C::kSpan >> 4) << 16));
            const uint32_t tm = uniform(tmem);
            // S at column col = Q K^T of the K tile in ring slot s, steps k0 to k1
            auto issue_s = [&](uint32_t col, uint32_t qtile, uint32_t s, int k0, int k1) {
                const uint32_t a = q_lo + qtile * (uint32_t)(C::kQTile >> 4), b = k_lo + s * (uint32_t)(C::kTile >> 4);
#pragma unroll
                for (int kk = k0; kk < k1; ++kk) {
                    const uint32_t h = (uint32_t)(kk >> 2), o = (uint32_t)(kk & 3) * 2u;
                    tc_mma(tm + col, sw128_desc_of(a + h * 1024u + o, sw128_desc_hi(1024)),
                           sw128_desc_of(b + h * (uint32_t)(C::kSpan >> 4) + o, kv_hi), kIdS, kk > 0 ? 1u : 0u);
                }
            };
            // O of stream t (+)= P V, P at column col, of the V tile in ring slot s
            auto issue_o = [&](uint32_t t, uint32_t col, uint32_t s, uint32_t acc) {
                const uint32_t b = v_lo + s * (uint32_t)(C::kTile >> 4);
#pragma unroll
                for (int part = 0; part < C::kParts; ++part)
#pragma unroll
                    for (int kk = 0; kk < KT / 16; ++kk)
                        tc_mma_ts(tm + 256u + t * (uint32_t)C::kOCols, tm + col + (uint32_t)(C::part_col(part) + kk * 8),
                                  sw128_desc_of(b + (uint32_t)kk * (uint32_t)(C::kGroup >> 3), kv_hi), kIdO, part > 0 || kk > 0 ? 1u : acc);
            };
            // ring places: d tiles on (d < S)
            struct Slot {
                uint32_t s, r;
                __device__ __forceinline__ Slot ahead(uint32_t d) const {
                    const bool wrap = s + d >= (uint32_t)S;
                    return Slot{wrap ? s + d - (uint32_t)S : s + d, wrap ? r ^ 1u : r};
                }
            };
            Slot at{0, 0};  // the next K tile; its V follows
            auto landed = [&](const Slot& x) { return (bool)__all_sync(0xffffffffu, mbar_test_wait(full((int)x.s), x.r)); };
            auto wait_slot = [&](const Slot& x) { wait(full((int)x.s), x.r); };
#pragma unroll 1
            while (next_segment(nseg, g)) {
                const int nt = (int)uniform((uint32_t)g.nt);
                // Every segment waits once for both O's of the one before it and then ends with
                // an arrival on seg_done, which every softmax warp waits for before it gives
                // the O's of this one back: so neither side is ever two phases ahead, also
                // where a stream has no tiles and nothing else holds its warps back.
                const uint32_t free_ph = (uint32_t)nseg & 1u;
                const bool parity = uniform((uint32_t)g.flags & 1u) != 0u;
                const int e0 = (int)uniform((uint32_t)g.e0);
                // Key tiles i = 0 .. nt - 1. S of a stream's next tile is issued right behind P V of
                // this one, which reads P where that S goes: the products run in the order of
                // their issue. The queue of the tensor cores holds two or three products of 64
                // cycles, so they run dry wherever this warp spends more than that between two:
                // the next tiles are looked for between the products of a batch (a look costs
                // 100 cycles), and what is left before P V is the wait for P.
                auto take_p = [&](int t) {
                    wait(p_full(t), (cnt >> t) & 1u);
                    cnt ^= 1u << t;
                };
                if (nt > 0) {
                    wait(q_full, (uint32_t)(nq & 1));
                    ++nq;
                }
                Slot v = at.ahead(1);
                if (NB == 3 && nt > 0) {
                    // Products k = 0 .. N - 1 (see Products): S of k + 3 goes where P of k was, right
                    // behind its P V.
                    const Products order{e0, nt, parity};
                    const int N = order.count();
                    int ks = 0;  // the next S, its K tile
                    Slot kt = at;
                    bool k_in = false, v_in = false;
                    auto next_s = [&]() {
                        const bool last = order.last_of_tile(ks);
                        if (!k_in) wait_slot(kt);
                        k_in = !last;
                        if (elect_one()) {
                            issue_s(C::place_col(sb), !parity && last ? 1u : 0u, kt.s, 0, D / 16);
                            tc_commit(s_full((int)sb));
                            if (last) tc_commit(empty((int)kt.s));
                            if (ks + 1 == N) tc_commit(q_empty);
                        }
                        __syncwarp();
                        if (last) kt = kt.ahead(2);
                        sb = sb == 2u ? 0u : sb + 1u;
                        ++ks;
                    };
                    while (ks < N && ks < 3) next_s();
                    wait(o_free(0), free_ph);
                    wait(o_free(1), free_ph);
                    int begun = 0;  // per stream (bit t): O holds something; float32: half of a pair of tiles
#pragma unroll 1
                    for (int k = 0; k < N; ++k) {
                        const bool last = order.last_of_tile(k);
                        const int t = order.stream(k, last);
                        if (!v_in) wait_slot(v);
                        v_in = !last;
                        wait(p_full((int)pb), pph);
                        if (elect_one()) {
                            issue_o((uint32_t)t, C::place_col(pb), v.s, (uint32_t)(begun >> t) & 1u);
                            tc_commit(o_done((int)pb));
                            if (last) tc_commit(empty((int)v.s));
                        }
                        __syncwarp();
                        begun = F32OUT ? begun ^ (1 << t) : begun | (1 << t);
                        if (ks < N) next_s();
                        if (last) v = v.ahead(2);
                        pph ^= pb == 2u ? 1u : 0u;
                        pb = pb == 2u ? 0u : pb + 1u;
                    }
                } else if (nt > 0 && !parity) {
                    // two row tiles: row tile 0 takes the first e0 key tiles, row tile 1 all
                    wait_slot(at);
                    if (elect_one()) {
                        if (e0 > 0) {
                            issue_s(0u, 0, at.s, 0, D / 16);
                            tc_commit(s_full(0));
                        }
                        issue_s(128u, 1, at.s, 0, D / 16);
                        tc_commit(s_full(1));
                        tc_commit(empty((int)at.s));
                        if (nt == 1) tc_commit(q_empty);
                    }
                    __syncwarp();
                    wait(o_free(0), free_ph);
                    wait(o_free(1), free_ph);
                    bool v_ok = false, k_ok = false;
                    Slot k = at.ahead(2);
#pragma unroll 1
                    for (int i = 0; i < nt; ++i) {
                        const bool more = i + 1 < nt;
                        if (!v_ok) wait_slot(v);
                        if (i < e0) {
                            take_p(0);
                            if (elect_one()) {
                                issue_o(0u, 0u, v.s, F32OUT ? (uint32_t)i & 1u : (i > 0 ? 1u : 0u));
                                if (F32OUT || i + 1 == e0) tc_commit(o_done(0));
                            }
                            __syncwarp();
                            if (i + 1 < e0) {
                                if (!k_ok) wait_slot(k);
                                k_ok = true;
                                if (elect_one()) {
                                    issue_s(0u, 0, k.s, 0, D / 16);
                                    tc_commit(s_full(0));
                                }
                                __syncwarp();
                            }
                        }
                        take_p(1);
                        if (elect_one()) {
                            issue_o(1u, 128u, v.s, F32OUT ? (uint32_t)i & 1u : (i > 0 ? 1u : 0u));
                            if (F32OUT || !more) tc_commit(o_done(1));
                            tc_commit(empty((int)v.s));
                        }
                        __syncwarp();
                        if (more) {
                            if (!k_ok) wait_slot(k);
                            if (elect_one()) issue_s(128u, 1, k.s, 0, D / 32);
                            __syncwarp();
                            const Slot v1 = v.ahead(2), k1 = k.ahead(2);
                            v_ok = landed(v1);
                            if (elect_one()) {
                                issue_s(128u, 1, k.s, D / 32, D / 16);
                                tc_commit(s_full(1));
                                tc_commit(empty((int)k.s));
                                if (i + 2 == nt) tc_commit(q_empty);
                            }
                            __syncwarp();
                            k_ok = i + 2 < nt && landed(k1);
                            v = v1;
                            k = k1;
                        }
                    }
                } else if (nt > 0) {
                    // one row tile: the streams take the key tiles in turn
                    auto first = [&](auto T, const Slot& x, bool last) {
                        constexpr int t = decltype(T)::value;
                        wait_slot(x);
                        if (elect_one()) {
                            issue_s(128u * t, 0, x.s, 0, D / 16);
                            tc_commit(s_full(t));
                            tc_commit(empty((int)x.s));
                            if (last) tc_commit(q_empty);
                        }
                        __syncwarp();
                    };
                    first(Stream<0>{}, at, nt == 1);
                    if (nt > 1) first(Stream<1>{}, at.ahead(2), nt == 2);
                    wait(o_free(0), free_ph);
                    wait(o_free(1), free_ph);
                    Slot k = at.ahead(4);
                    auto advance = [&](auto T, int i) {
                        constexpr int t = decltype(T)::value;
                        const bool more = i + 2 < nt;
                        wait_slot(v);
                        take_p(t);
                        if (elect_one()) {
                            issue_o(t, 128u * t, v.s, F32OUT ? (uint32_t)(i >> 1) & 1u : (i >= 2 ? 1u : 0u));
                            if (F32OUT || !more) tc_commit(o_done(t));
                            tc_commit(empty((int)v.s));
                        }
                        __syncwarp();
                        if (more) first(T, k, i + 3 == nt);
                        v = v.ahead(2);
                        k = k.ahead(2);
                    };
#pragma unroll 1
                    for (int i = 0; i < nt; i += 2) {
                        advance(Stream<0>{}, i);
                        if (i + 1 < nt) advance(Stream<1>{}, i + 1);
                    }
                } else {
                    wait(o_free(0), free_ph);
                    wait(o_free(1), free_ph);
                }
                const uint32_t end = at.s + 2u * (uint32_t)nt + (staged(g) ? 2u : 0u);
                at.r ^= (end / (uint32_t)S) & 1u;
                at.s = end % (uint32_t)S;
                if (elect_one()) tc_commit(seg_done);
                __syncwarp();
            }
            if (lane == 0) {
                if (*s_abort != 0) give_up();
                tc_commit(done);  // every product issued above has finished once this arrives
                mbar_wait_drain(done, 0u);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        uint32_t tS = tmem + lane_off + (uint32_t)(t * 128);
        const uint32_t tO = tmem + lane_off + 256u, tOt = tO + (uint32_t)(t * C::kOCols);
        const int rtok = r / p.G, rhead = r - rtok * p.G, stok = lane / p.G, shead = lane - stok * p.G;
        const uint64_t qscale2 = pack2(p.qscale, p.qscale);
        float ref_low = 0.f, ref_high = 0.f;
        if constexpr (fixed) {
            ref_low = p.ref_low;
            ref_high = p.ref_high;
        }
        uint32_t cnt = 0, odc[2] = {0, 0}, nx = 0, ring = 0;  // tiles, o_done's, exchanges, ring tiles so far
        uint32_t nd = 0;                                      // segments done
        uint32_t kb = 0;                                      // three places: products so far
#pragma unroll 1
        for (bool more = next_segment(nseg, g); more; ++nd) {
            const bool parity = (g.flags & 1) != 0, whole = (g.flags & 2) != 0, spread = (g.flags & 4) != 0;
            const int hd = spread ? shead : rhead;
            const int ltok = spread ? stok : (parity ? 0 : t * p.TQ) + rtok;  // token of this row within the item
            const bool valid = (spread ? stok < p.TS : rtok < p.TQ) && ltok < g.tokens;
            // Keys that this row sees, and the fewest of the warp's rows. With three places the
            // softmax is what a tile waits for: no votes a tile, and rows of no token go unmasked
            // (16,384 tokens, d 64: 1140 -> 1106 us; with two places and d 128 337 -> 341, float32
            // 283 -> 300, so the votes stay there).
            const int kmax = valid ? min(g.nk, max(EX ? g.prefix : 0, g.kfirst + ltok + 1)) : (NB == 3 || shaped ? INT_MAX : 0);
            const int kmin = __reduce_min_sync(0xffffffffu, kmax);
            // with score options: the first key of the item's last token, and of this row; the row's slope
            const int klast = EX ? (window.keys > 0 ? max(g.first, g.kfirst + g.tokens - window.keys) : g.first) : 0;
            auto first_key = [&]() {
                return !valid ? 0 : window.keys > 0 ? max(g.first, g.kfirst + ltok + 1 - window.keys) : g.first;
            };
            float slope = 0.f;
            if constexpr (MODE == kShaped) {
                if (valid && p.slopes != nullptr) slope = p.slopes[g.head * p.G + hd] * 1.4426950408889634f;
            }
            // which of the columns col, col + 1, .. (32 at most) of key tile j the row sees
            auto seen_of = [&](int lim, int j, int col) {
                return column_bits(klast > j * KT ? first_key() - j * KT - col : 0, lim - col);
            };
            auto mask = [&](auto& x, int lim, int j, int col) {
                if constexpr (shaped) mask_bits(x, seen_of(lim, j, col));
                else mask_columns(x, lim - col);
            };
            // shaped scores less sub of columns col, col + 1, .. of key tile j; `part`: some row of the warp does not
            // see all of the tile
            auto shape = [&](auto& x, int lim, int j, int col, bool part, float sub) {
                if constexpr (shaped) {
                    const int from = j * KT + col - (g.kfirst + ltok);
                    uint32_t seen = ~0u;
                    float mine = 0.f;
                    if (part) seen = seen_of(lim, j, col);
                    if (!BACK || p.cap != 0.f) mine = part ? magnitude(x, seen) : magnitude(x);
                    mine = valid ? mine : 0.f;
                    shape_scores<F32OUT, BACK>(x, p, slope, (float)from, g.prefix > g.kfirst + 1 && (j + 1) * KT - 1 > g.kfirst, mine, sub);
                    if (part) mask_bits(x, seen);
                }
            };
            const bool any = __any_sync(0xffffffffu, valid);
            const int st0 = parity ? (g.nt + 1) >> 1 : g.e0, st1 = parity ? g.nt >> 1 : g.nt;
            const int nt = t == 0 ? st0 : st1;
            const int jstep = (parity ? 2 : 1) * (BACK ? -1 : 1);
            float m = fixed ? ref_low : -INFINITY, l = 0.f;
            float acc[F32OUT ? D : 1];  // float32 output: O is added up here, tile by tile
            if constexpr (F32OUT) {
#pragma unroll
                for (int k = 0; k < D; ++k) acc[k] = 0.f;
            }
            auto add_o = [&]() {
                if constexpr (F32OUT) {
#pragma unroll
                    for (int cc = 0; cc < D; cc += 32) {
                        uint32_t o[32];
                        tmem_ld32(tOt + (uint32_t)cc, o);
                        tmem_landed(o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) acc[cc + k] += __uint_as_float(o[k]);
                    }
                }
            };
            // The V tile that may hold rows past the last key. They become zeros (what lies
            // there may be no number, and its weight of 0 would not help): by the first stream
            // that uses them, before its P is full.
            const int jlast = g.jb + g.nt - 1;
            const bool clears = g.kend < (jlast + 1) * KT && (t == 0 || parity || jlast >= g.jb + st0);
            // (the same before the first key that the item sees)
            const bool clears_low = EX && g.begins != 0 && g.kbegin > g.jb * KT && (t == 0 || parity || st0 == 0);
            int j = BACK ? jlast - (parity ? t : 0) : (parity ? g.jb + t : g.jb);
            // three places: the number of the product of a stream's tile i; whether it has finished
            // P V. A barrier that has gone on by two phases looks like one that has not moved, so
            // product k + 3 must not finish before a warp has found k: before a stream's last
            // tile it comes behind a product that waits for the stream's P; behind it, see below.
            const Products order{g.e0, g.nt, parity};
            auto product = [&](int tt, int i) { return kb + (uint32_t)order.of(tt, i); };
            auto wait_o = [&](uint32_t k) { wait(o_done((int)(k % 3u)), (k / 3u) & 1u); };
#pragma unroll 1
            for (int i = 0; i < nt; ++i, j += jstep) {
                const int lim = kmax - j * KT;  // columns of this tile the row sees
                const bool part = (NB == 3 ? kmin - j * KT < KT : (bool)__any_sync(0xffffffffu, lim < KT)) || (shaped && klast > j * KT);
                if (NB == 2 && aborted()) break;
                // O holds two tiles at most (24 steps of the accumulator)
                bool take_o = F32OUT && i > 0 && (i & 1) == 0;
                int place = t;
                if constexpr (NB == 3) {
                    const uint32_t k = product(t, i), b = k % 3u;
                    place = (int)b;
                    tS = tmem + lane_off + C::place_col(b);
                    wait(s_full(place), (k / 3u) & 1u);
                } else {
                    if (take_o) {
                        wait(o_done(t), (cnt - 1u) & 1u);
                        if (any) add_o();
                        take_o = false;
                    }
                    wait(s_full(t), cnt & 1u);
                }
                if constexpr (MODE == kMasked) {
                    // Scores that are only scaled are masked where they lie: in an item's first tiles alone, so in
                    // a loop that is short rather than in the code of all tiles.
                    if (any && klast > j * KT) {
                        const int low = first_key() - j * KT;
#pragma unroll 1
                        for (int cc = 0; cc < KT; cc += 16) {
                            uint32_t x[16];
                            tmem_ld16(tS + (uint32_t)cc, x);
                            tmem_landed(x);
                            mask_before(x, low - cc);
                            tmem_st16(tS + (uint32_t)cc, x);
                        }
                        tmem_wait_st();
                    }
                }
                if (any) {
                    // The reference grows to mx: what was added up shrinks by a. With two places S of
                    // this tile came behind the products of the tiles before, so O holds those.
                    auto grow_to = [&](float mx, bool grow) {
                        if (NB == 3 && i > 0) wait_o(product(t, i - 1));
                        const float a = !grow ? 1.f : shaped ? whole_power(m - mx) : ex2((m - mx) * p.qscale);  // 0 from -inf
                        l *= a;
                        if (grow) m = mx;
                        if constexpr (F32OUT) {
                            if (take_o) {
                                add_o();
                                take_o = false;
                            }
                            if ((i & 1) != 0) {
                                add_o();
                                const uint32_t zero[32] = {};
#pragma unroll 1
                                for (int cc = 0; cc < D; cc += 32) tmem_st32(tOt + (uint32_t)cc, zero);
                            }
#pragma unroll
                            for (int k = 0; k < D; ++k) acc[k] *= a;
                        } else if (i > 0) {
#pragma unroll 1
                            for (int cc = 0; cc < D; cc += 32) {
                                uint32_t o[32];
                                tmem_ld32(tOt + (uint32_t)cc, o);
                                tmem_landed(o);
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                                tmem_st32(tOt + (uint32_t)cc, o);
                            }
                        }
                        return a;
                    };
                    // Shaped scores come less the reference as it is. It moves where their maximum `top` (less it
                    // as well) asks for that; a constant one is set where a row sees its first keys.
                    // Returns by how much, with what is to be scaled meanwhile done by scale(a). It moves by a
                    // whole number, so a is a power of 2: the tile's weights are in bf16 parts by then, and would be
                    // rounded again (three parts to those of one). Those of float32 results are whole
                    // from the start, where the move is exact; of bf16 weights the largest is 1, which is.
                    const bool looks = !fixed || (bool)__any_sync(0xffffffffu, valid && l == 0.f && lim > 0 && first_key() < (j + 1) * KT);
                    bool none = l == 0.f;
                    auto settle = [&](float top, auto&& scale) {
                        const float sub = m == -INFINITY ? 0.f : m;
                        bool moves = top != -INFINITY && (fixed ? none : m == -INFINITY || top > kShapedRescale);
                        moves = moves && valid;
                        none = none && top == -INFINITY;
                        if (!__any_sync(0xffffffffu, moves)) return 0.f;
                        const float to = fixed ? fminf(fmaxf(sub + top, ref_low), ref_high)
                                               : sub + (F32OUT || m != -INFINITY ? ceilf(top) : top);
                        if constexpr (fixed) {
                            if (moves) m = to;
                        } else {
                            scale(grow_to(to, moves));
                        }
                        return moves ? sub - to : 0.f;
                    };
                    // A constant reference where rows see their first keys: the cap of their largest product of
                    // this tile. (Weights are rounded to bf16, and a row's largest is exact where it is 1.) A pass
                    // over the products before the tile takes the short path: 24 prompts of 1,000 tokens 268 -> 257 us;
                    // in the kernel for long items it costs the others' code its place (16,384 tokens 1,574 -> 1,640).
                    auto begin_fixed = [&](auto& x) {
                        constexpr int W = sizeof(x) / 4;
                        float top = -INFINITY;
#pragma unroll 1
                        for (int cc = 0; cc < KT; cc += W) {
                            tmem_load(tS + (uint32_t)cc, x);
                            tmem_landed(x);
                            if (part) mask(x, lim, j, cc);
                            top = max_of(x, top);
                        }
                        if constexpr (fixed) {
                            if (valid && none && top != -INFINITY) m = fminf(fmaxf(cap_of(top, p), ref_low), ref_high);
                        }
                    };
                    // biased scores: whether the tile's keys all lie on one side of the rows, which have seen keys;
                    // a row's bias at the tile's first column, less the reference
                    auto fast_ok = [&](bool part) {
                        return !part && !(g.prefix > g.kfirst + 1 && (j + 1) * KT - 1 > g.kfirst) &&
                               !__any_sync(0xffffffffu, valid && m == -INFINITY);
                    };
                    auto fast_row = [&]() { return fmaf(slope, (float)(j * KT - (g.kfirst + ltok)), m == -INFINITY ? 0.f : -m); };
                    auto shift = [&](auto& x, float by) {
                        each_pair(x, [&](uint64_t v) { return add2(v, pack2(by, by)); });
                    };
                    if (spread) {
                        // this warp's quarter of the columns; P of the others is 0 in its rows
                        constexpr int Q = KT / 4;
                        const int w = warp & 3;
                        uint32_t x[Q];
                        tmem_load(tS + (uint32_t)(w * Q), x);
                        tmem_landed(x);
                        if constexpr (shaped) {
                            shape(x, lim, j, w * Q, part, m == -INFINITY ? 0.f : m);
                            if (looks) {
                                const float by = settle(max_of(x, -INFINITY), [](float) {});
                                if (__any_sync(0xffffffffu, by != 0.f)) shift(x, by);
                            }
                        } else {
                            if (part) mask(x, lim, j, w * Q);
                            const float mx = max_of(x, m);
                            const bool grow = (NB == 2 || valid) && (mx - m) * p.qscale > kRescale;  // false where both are -inf
                            if (__any_sync(0xffffffffu, grow)) grow_to(mx, grow);
                        }
                        const float sub = shaped || m == -INFINITY ? 0.f : m * p.qscale;
                        if constexpr (F32OUT) {
                            uint32_t q[3][8];
                            l += parts16<16, shaped>(x, p.qscale, sub, q);
#pragma unroll
                            for (int e = 0; e < 3; ++e) {
                                const uint32_t zero[8] = {};
#pragma unroll
                                for (int v = 0; v < 4; ++v) {
                                    if (v == w) tmem_st8(tS + (uint32_t)(C::part_col(e) + 8 * v), q[e]);
                                    else tmem_st8(tS + (uint32_t)(C::part_col(e) + 8 * v), zero);
                                }
                            }
                        } else {
                            uint64_t sum[2] = {0, 0};
                            uint32_t q[16];
                            const uint32_t zero[16] = {};
                            weights32<shaped>(x, qscale2, pack2(-sub, -sub), q, sum);
#pragma unroll
                            for (int v = 0; v < 4; ++v) {
                                if (v == w) tmem_st16(tS + (uint32_t)(16 * v), q);
                                else tmem_st16(tS + (uint32_t)(16 * v), zero);
                            }
                            float a, b;
                            unpack2(add2(sum[0], sum[1]), a, b);
                            l += a + b;
                        }
                    } else if constexpr (F32OUT) {
                        if constexpr (!shaped) {
                            float mx = m;
                            {
                                uint32_t x[64];
                                tmem_ld64(tS, x);
                                tmem_landed(x);
                                if (part) mask(x, lim, j, 0);
                                mx = max_of(x, mx);
                            }
                            const bool grow = (NB == 2 || valid) && (mx - m) * p.qscale > kRescale;  // false where both are -inf
                            if (__any_sync(0xffffffffu, grow)) grow_to(mx, grow);
                        }
                        float sub = m == -INFINITY ? 0.f : m * p.qscale;
                        int cc = 0;
                        if constexpr (shaped) {
                            const uint32_t part_at[3] = {(uint32_t)C::part_col(0), (uint32_t)C::part_col(1), (uint32_t)C::part_col(2)};
                            if constexpr (fixed) {
                                if (looks) {
                                    uint32_t x[16];
                                    begin_fixed(x);
                                }
                                if (!part) cc = fast_parts<true, false>(tS, part_at, p, -m, 0.f, valid, l);
                            } else if (fast_ok(part)) {
                                const float row = fast_row();
                                cc = p.cap != 0.f ? fast_parts<true, true>(tS, part_at, p, row, slope, valid, l)
                                                  : fast_parts<false, true>(tS, part_at, p, row, slope, valid, l);
                            }
                        }
#pragma unroll 1
                        for (; cc < 64; cc += 16) {
                            uint32_t x[16], q[3][8];
                            tmem_load(tS + (uint32_t)cc, x);
                            tmem_landed(x);
                            if constexpr (shaped) {
                                shape(x, lim, j, cc, part, m == -INFINITY ? 0.f : m);
                                if constexpr (!fixed) {
                                    const float by = settle(max_of(x, -INFINITY), [&](float a) {
                                        tmem_wait_st();
#pragma unroll 1
                                        for (int c = 0; c < cc / 2; c += 8)
#pragma unroll
                                            for (int e = 0; e < 3; ++e) scale_pairs8(tS + (uint32_t)(C::part_col(e) + c), a);
                                    });
                                    if (__any_sync(0xffffffffu, by != 0.f)) shift(x, by);
                                }
                            } else if (part) {
                                mask(x, lim, j, cc);
                            }
                            l += parts16<16, shaped>(x, p.qscale, sub, q);
                            // the third part goes over columns of S that have been read: 8 for 16
#pragma unroll
                            for (int e = 0; e < 3; ++e) tmem_st8(tS + (uint32_t)(C::part_col(e) + cc / 2), q[e]);
                        }
                    } else {
                        uint64_t sum[2] = {0, 0};
                        uint32_t w[16];
                        if constexpr (shaped) {
                            int cc = 0;
                            if constexpr (MODE == kCapped) {
                                if (looks) {
                                    uint32_t x[32];
                                    begin_fixed(x);
                                }
                                if (!part) cc = fast_tile<true, false, 1>(tS, p, -m, 0.f, valid, sum);
                            } else if constexpr (MODE == kCappedLong) {
                                if (!part && !looks) cc = fast_tile<true, false, 4>(tS, p, -m, 0.f, valid, sum);
                            } else if (fast_ok(part)) {
                                const float row = fast_row();
                                cc = p.cap != 0.f ? fast_tile<true, true, 1>(tS, p, row, slope, valid, sum)
                                                  : fast_tile<false, true, 1>(tS, p, row, slope, valid, sum);
                            }
                            // the rest, in any case
#pragma unroll 1
                            for (; cc < 128; cc += 32) {
                                uint32_t x[32];
                                tmem_ld32(tS + (uint32_t)cc, x);
                                tmem_landed(x);
                                shape(x, lim, j, cc, part, m == -INFINITY ? 0.f : m);
                                if (MODE != kCapped && looks) {
                                    const float by = settle(max_of(x, -INFINITY), [&](float a) {
                                        sum[0] = mul2(sum[0], pack2(a, a));
                                        sum[1] = mul2(sum[1], pack2(a, a));
                                        tmem_wait_st();
#pragma unroll 1
                                        for (int c = 0; c < cc / 2; c += 8) scale_pairs8(tS + (uint32_t)c, a);
                                    });
                                    if (__any_sync(0xffffffffu, by != 0.f)) shift(x, by);
                                }
                                weights32<true>(x, 0, 0, w, sum);
                                tmem_st16(tS + (uint32_t)(cc >> 1), w);
                            }
                        } else {
                            uint32_t x0[64], x1[64];
                            tmem_ld64(tS, x0);
                            tmem_landed(x0);
                            tmem_ld64(tS + 64u, x1);
                            if (part) mask(x0, lim, j, 0);
                            float mx = max_of(x0, m);
                            tmem_landed(x1);
                            if (part) mask(x1, lim, j, 64);
                            mx = max_of(x1, mx);
                            const bool grow = (NB == 2 || valid) && (mx - m) * p.qscale > kRescale;  // false where both are -inf
                            if (__any_sync(0xffffffffu, grow)) grow_to(mx, grow);
                            const float sub = m == -INFINITY ? 0.f : m * p.qscale;
                            const uint64_t nsub2 = pack2(-sub, -sub);
                            weights32(x0, qscale2, nsub2, w, sum);
                            tmem_st16(tS, w);
                            weights32(x0 + 32, qscale2, nsub2, w, sum);
                            tmem_st16(tS + 16u, w);
                            weights32(x1, qscale2, nsub2, w, sum);
                            tmem_st16(tS + 32u, w);
                            weights32(x1 + 32, qscale2, nsub2, w, sum);
                            tmem_st16(tS + 48u, w);
                        }
                        float a, b;
                        unpack2(add2(sum[0], sum[1]), a, b);
                        l += a + b;
                    }
                }
                if (NB == 3 && take_o) {  // before P V of this tile overwrites it
                    wait_o(product(t, i - 1));
                    if (any) add_o();
                }
                ++cnt;
                const bool low = EX && clears_low && j == g.jb;
                if ((clears && j == jlast) || low) {
                    const uint32_t k = ring + 2u * (uint32_t)(BACK ? jlast - j : j - g.jb) + 1u, s = k % (uint32_t)S;
                    wait(full((int)s), (k / (uint32_t)S) & 1u);
                    uint8_t* tile = s_raw + 2 * C::kQTile + s * C::kTile;
                    // rows [0, n0) and [rows, KT)
                    const int n0 = low ? g.kbegin - g.jb * KT : 0;
                    const int rows = clears && j == jlast ? g.kend - jlast * KT : KT, chunks = (n0 + KT - rows) * 8;
#pragma unroll 1
                    for (int e = r; e < chunks * C::kHalves; e += 128) {
                        const int h = e >= chunks ? 1 : 0, c = e - h * chunks, y = (c >> 3) < n0 ? (c >> 3) : rows - n0 + (c >> 3);
                        *reinterpret_cast<uint4*>(tile + h * C::kSpan + (y >> 3) * C::kGroup + (y & 7) * 128 + (c & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_async_shared();
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(place));
            }
            ring += 2u * (uint32_t)g.nt;
            // the next segment, while the products run (float32: there are no registers for it)
            Segment gn;
            if (!F32OUT) more = next_segment(nseg, gn);
            // o_done: every tile with a float32 output, else a stream's last one
            odc[0] += F32OUT ? (uint32_t)st0 : (st0 > 0 ? 1u : 0u);
            odc[1] += F32OUT ? (uint32_t)st1 : (st1 > 0 ? 1u : 0u);
            if (NB == 3) {
                // Nothing of row tile 0 holds back what comes behind its last product. Where a product
                // of this segment uses that place again (128 tokens a row tile and tiles of 64
                // keys: float32, one head per KV head), it waits for the segment's end instead;
                // elsewhere the place's next product is one of the next segment, which
                // waits for both streams' O.
                if (F32OUT && order.lapped(t)) wait(seg_done, nd & 1u);
                else if (nt > 0) wait_o(product(t, nt - 1));
            } else if (nt > 0) {
                wait(o_done(t), (odc[t] - 1u) & 1u);
            }
            if constexpr (F32OUT) {
                // the whole O goes where the rest reads it
                if (nt > 0) {
                    if (any) {
                        add_o();
#pragma unroll
                        for (int cc = 0; cc < D; cc += 32) {
                            uint32_t o[32];
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(acc[cc + k]);
                            tmem_st32(tOt + (uint32_t)cc, o);
                        }
                        tmem_wait_st();
                    }
                    tc_fence_before();
                }
            }
            // row of out / lse, or of this CTA's part of the item
            const int64_t row = whole ? (int64_t)(g.row0 + ltok) * p.Hq + g.head * p.G + hd
                                      : (int64_t)(2 * blockIdx.x + (g.begins ? 1 : 0)) * p.slot_rows + (parity ? r : t * 128 + r);
            float ca = 1.f, cb = 0.f;          // factors of O0 (or of this stream's O) and O1
            uint32_t oa = tOt;
            int col0 = 0, cols = D;
            const bool have = parity ? st0 > 0 : nt > 0, both = parity && st1 > 0;
            if (parity) {
                if (st0 > 0) {
                    // the other stream: all but its last product came before ours
                    if (t == 1 || st1 > 0) {
                        if (NB == 3) wait_o(product(t ^ 1, (t == 0 ? st1 : st0) - 1));
                        else wait(o_done(t ^ 1), (odc[t ^ 1] - 1u) & 1u);
                    }
                    s_ml[t * 128 + r] = make_float2(m, l);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(x_bar);
                    wait(x_bar, nx & 1u);
                    ++nx;
                    const float2 A = s_ml[r], B = s_ml[128 + r];
                    m = fmaxf(A.x, B.x);
                    const float ms = m == -INFINITY ? 0.f : m;
                    ca = ex2((A.x - ms) * p.qscale);
                    cb = ex2((B.x - ms) * p.qscale);
                    l = A.y * ca + B.y * cb;
                }
                oa = tO;
                col0 = t * (D / 2);
                cols = D / 2;
            }
            if (whole) {
                const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
                ca *= inv;
                cb *= inv;
            }
            const bool put = staged(g), box = put && (t == 0 || g.tokens == t2);
            const uint32_t kput = ring + (uint32_t)t, sput = kput % (uint32_t)S;
            // (Also without a box to put there: stream 1's slot comes at least five tiles behind
            // the first slot of the staged item before, so it is free only once that item's rows
            // have been sent, and staged_full cannot complete a second phase before the
            // Q warp has found the first.)
            if (put) wait(empty((int)sput), ((kput / (uint32_t)S) & 1u) ^ 1u);
            if (box) {
                const uint32_t s = sput;
                uint8_t* tile = s_raw + 2 * C::kQTile + s * C::kTile + r * 128;
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 32) {
                    uint32_t o[32] = {};
                    if (have) {
                        tmem_ld32(oa + (uint32_t)cc, o);
                        tmem_landed(o);
                    }
                    const int h = (cc >> 6) * 16384, c0 = (cc & 63) >> 3;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_bf16(__uint_as_float(o[8 * q + 2 * e]) * ca, __uint_as_float(o[8 * q + 2 * e + 1]) * ca);
                        *reinterpret_cast<uint4*>(tile + h + (((c0 + q) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                fence_async_shared();
                if (valid) p.lse[row] = l == 0.f ? -INFINITY : fmaf(m, p.qscale, log2f(l)) * 0.6931471805599453f;
            } else if (any) {
                // one warp's rows: their stores are few, the exchange would be code to fetch (1,000
                // decodes over 100 to 500 keys: 462 -> 454 us)
                const bool few = parity && g.tokens <= p.TS;
                const RowPair rows = pair_rows(whole ? reinterpret_cast<char*>(p.out) + row * (D * (F32OUT ? 4 : 2))
                                                     : reinterpret_cast<char*>(p.part_o) + row * (D * 4), valid, lane);
                // W columns of O (both streams' where there are two), scaled
                auto take = [&](int cc, auto& o) {
                    constexpr int W = sizeof(o) / 4;
#pragma unroll
                    for (int k = 0; k < W; ++k) o[k] = 0u;
                    if (have) {
                        tmem_load(oa + (uint32_t)cc, o);
                        tmem_landed(o);
#pragma unroll
                        for (int k = 0; k < W; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * ca);
                    }
                    if (both) {
                        uint32_t o1[W];
                        tmem_load(tO + (uint32_t)(C::kOCols + cc), o1);
                        tmem_landed(o1);
#pragma unroll
                        for (int k = 0; k < W; ++k)
                            o[k] = __float_as_uint(fmaf(__uint_as_float(o1[k]), cb, __uint_as_float(o[k])));
                    }
                };
                // (in short loops: run once for an item, their code is not in the cache)
                if (!F32OUT && whole) {
#pragma unroll 1
                    for (int cc = col0; cc < col0 + cols; cc += 32) {
                        uint32_t o[32], w[16];
                        take(cc, o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) w[k] = pack_bf16(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
                        if (few) {
                            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<char*>(p.out) + row * (D * 2) + cc * 2);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (valid) dst[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
                        } else {
                            store_rows(w, rows, cc * 2, p.out_align32);
                        }
                    }
                } else {
#pragma unroll 1
                    for (int cc = col0; cc < col0 + cols; cc += 16) {
                        uint32_t o[16];
                        take(cc, o);
                        store_rows(o, rows, cc * 4, !whole || p.out_align32);
                    }
                }
                if (valid && (!parity || t == 0)) {
                    if (whole)
                        p.lse[row] = l == 0.f ? -INFINITY : fmaf(m, p.qscale, log2f(l)) * 0.6931471805599453f;
                    else
                        p.part_ml[row] = make_float2(m, l);
                }
            }
            kb += (uint32_t)order.count();
            if (put) {
                ring += 2u;
                __syncwarp();
                if (lane == 0) mbar_arrive(staged_full);
            }
            tc_fence_before();
            wait(seg_done, nd & 1u);
            if (lane == 0) {
                // eight arrivals each: four warps twice, or all eight once
                mbar_arrive(o_free(parity ? 0 : t));
                mbar_arrive(o_free(parity ? 1 : t));
            }
            if (F32OUT) more = next_segment(nseg, g);
            else g = gn;
        }
        if (lane == 0 && *s_abort != 0) give_up();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the parts of every item that spans CTAs, in order: grid (CTA in which an item
// may begin, slices of its rows), one pass with a running maximum. Latency is most of what
// it costs, so loads of several parts and rows are in flight: a warp takes two rows and four
// parts at a time; where each warp of a stream left parts (32 rows at most, up to 600
// parts), a CTA takes a row and its eight warps share the parts. 2.7 us
// behind a decode step, 7 to 10 us where every CTA left two parts of 256 rows (40 MB
// through L2); with 8 or 32 slices the same within 2 %.
constexpr int kMergeSlices = 16;
template <int D>
struct Joined {
    static constexpr int E = D / 32;
    float m = -INFINITY, l = 0.f, acc[E] = {};
    // n <= 4 parts more: their (m, l), and this lane's columns of their O
    __device__ __forceinline__ void add(const float2 (&ml)[4], const float (&v)[4][E], float qscale) {
        const float mx = fmaxf(fmaxf(fmaxf(m, ml[0].x), fmaxf(ml[1].x, ml[2].x)), ml[3].x);
        const float ms = mx == -INFINITY ? 0.f : mx, a = ex2((m - ms) * qscale);
        m = mx;
        l *= a;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= a;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float w = ex2((ml[u].x - ms) * qscale);  // 0 behind the last part
            l = fmaf(ml[u].y, w, l);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(v[u][e], w, acc[e]);
        }
    }
};

template <int D, bool F32OUT>
__global__ void __launch_bounds__(256) k_packed_merge(const PackedParams p) {
    constexpr int E = D / 32;
    __shared__ float s_acc[8][D];
    __shared__ float2 s_ml[8];
    pdl_wait();
    pdl_launch_dependents();
    const SplitItem d = p.items[blockIdx.x];
    if (d.parts <= 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool spread = d.tokens < 0;
    const int tokens = spread ? -d.tokens : d.tokens, rows = tokens * p.G, parts = spread ? 4 * d.parts : d.parts;
    const bool two = tokens > p.TQ;
    // row i of the item in part k
    auto at = [&](int i, int k) {
        const int tok = i / p.G, row = two && tok >= p.TQ ? 128 + i - p.TQ * p.G : i, c = spread ? k >> 2 : k;
        return (int64_t)(2 * (blockIdx.x + c) + (c == 0 ? 1 : 0)) * p.slot_rows + row + (spread ? (k & 3) * 32 : 0);
    };
    // parts k, k + ks, .. of row i (n of the four there are)
    auto fetch = [&](int i, int k, int ks, float2 (&ml)[4], float (&v)[4][E]) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool in = k + u * ks < parts;
            ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = 0.f;
            if (in) {
                const int64_t a = at(i, k + u * ks);
                ml[u] = p.part_ml[a];
                const float* o = p.part_o + a * D + lane * E;
                if constexpr (E == 4) {
                    const float4 f = *reinterpret_cast<const float4*>(o);
                    v[u][0] = f.x, v[u][1] = f.y, v[u][2] = f.z, v[u][3] = f.w;
                } else {
                    const float2 f = *reinterpret_cast<const float2*>(o);
                    v[u][0] = f.x, v[u][1] = f.y;
                }
            }
        }
    };
    auto finish = [&](int i, const Joined<D>& x) {
        const int tok = i / p.G, h = i - tok * p.G;
        const float inv = x.l > 0.f ? 1.f / x.l : (x.l == 0.f ? 0.f : x.l);
        const int64_t orow = (int64_t)(d.row0 + tok) * p.Hq + d.head * p.G + h;
        if (F32OUT) {
            float* o = reinterpret_cast<float*>(p.out) + orow * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(o + e) = make_float2(x.acc[e] * inv, x.acc[e + 1] * inv);
        } else {
            uint32_t* o = reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(p.out) + orow * D + lane * E);
#pragma unroll
            for (int e = 0; e < E; e += 2) o[e / 2] = pack_bf16(x.acc[e] * inv, x.acc[e + 1] * inv);
        }
        if (lane == 0) p.lse[orow] = x.l == 0.f ? -INFINITY : fmaf(x.m, p.qscale, log2f(x.l)) * 0.6931471805599453f;
    };
    if (spread) {
        for (int i = blockIdx.y; i < rows; i += kMergeSlices) {
            Joined<D> x;
            for (int k = warp; k < parts; k += 32) {
                float2 ml[4];
                float v[4][E];
                fetch(i, k, 8, ml, v);
                x.add(ml, v, p.qscale);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = x.acc[e];
            if (lane == 0) s_ml[warp] = make_float2(x.m, x.l);
            __syncthreads();
            if (warp == 0) {
                Joined<D> y;
#pragma unroll
                for (int w = 0; w < 8; w += 4) {
                    float2 ml[4];
                    float v[4][E];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        ml[u] = s_ml[w + u];
#pragma unroll
                        for (int e = 0; e < E; ++e) v[u][e] = s_acc[w + u][lane * E + e];
                    }
                    y.add(ml, v, p.qscale);
                }
                finish(i, y);
            }
            __syncthreads();
        }
    } else {
        constexpr int step = kMergeSlices * 8;
        for (int i = blockIdx.y * 8 + warp; i < rows; i += 2 * step) {
            const bool both = i + step < rows;
            Joined<D> x, y;
            for (int k = 0; k < parts; k += 4) {
                float2 ml[4], ml2[4];
                float v[4][E], v2[4][E];
                fetch(i, k, 1, ml, v);
                if (both) fetch(i + step, k, 1, ml2, v2);
                x.add(ml, v, p.qscale);
                if (both) y.add(ml2, v2, p.qscale);
            }
            finish(i, x);
            if (both) finish(i + step, y);
        }
    }
}

template <int D, bool F32OUT, bool FOLD, int MODE>
cudaError_t launch_t(const Params<(MODE != kPlain)>& p, const PackedMaps& m, int grid, bool merge, cudaStream_t st) {
    using C = AttCfg<D, F32OUT, FOLD>;
    cudaError_t e =
        cudaFuncSetAttribute(k_packed_att<D, F32OUT, FOLD, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_ex(k_packed_att<D, F32OUT, FOLD, MODE>, dim3((unsigned)grid), dim3(kAttThreads), C::kSmem, st, true, m.q, m.qs, m.k, m.v, m.o, p);
    if (e != cudaSuccess || !merge) return e;
    return launch_ex(k_packed_merge<D, F32OUT>, dim3((unsigned)grid, kMergeSlices), dim3(256), 0, st, true, static_cast<const PackedParams&>(p));
}

template <int MODE>
cudaError_t launch(const Params<(MODE != kPlain)>& p, const PackedMaps& m, int d, bool f32_out, int grid, bool merge, cudaStream_t st) {
    if (d == 64) return f32_out ? launch_t<64, true, false, MODE>(p, m, grid, merge, st) : launch_t<64, false, false, MODE>(p, m, grid, merge, st);
    if (p.kv_fold) return f32_out ? launch_t<128, true, true, MODE>(p, m, grid, merge, st) : launch_t<128, false, true, MODE>(p, m, grid, merge, st);
    return f32_out ? launch_t<128, true, false, MODE>(p, m, grid, merge, st) : launch_t<128, false, false, MODE>(p, m, grid, merge, st);
}
// For d = 128 and bf16 outputs.
template <int MODE>
cudaError_t launch_128(const Params<(MODE != kPlain)>& p, const PackedMaps& m, int grid, bool merge, cudaStream_t st) {
    return p.kv_fold ? launch_t<128, false, true, MODE>(p, m, grid, merge, st) : launch_t<128, false, false, MODE>(p, m, grid, merge, st);
}

}  // namespace

}  // namespace ha
