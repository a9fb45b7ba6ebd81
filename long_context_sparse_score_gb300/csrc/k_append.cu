// Append new tokens to a paged KV cache, rotating queries and keys by their
// positions on the way.
//
// k_append: token i of sequence s (nq new tokens, nk tokens once they are in)
// sits at position pos = nk - nq + i, in row pos % page_size of page
// table[s][pos / page_size]. Its queries and keys are rotated: pair p of the
// first `rot` dims, (x_p, x_{p + rot/2}) or, interleaved, (x_{2p}, x_{2p+1}),
// turns by the angle pos * inv_freq[p]; the other dims and the values are copied. With
// several axes (AXES) the angle is positions[axis[p]] * inv_freq[p] instead: a lane holds
// one axis' position and the others take it from there, so it costs one load a warp,
// beside those of the place.
//
// The angle in turns, pos * inv_freq / 2 pi, is kept as a 64-bit fixed-point
// fraction: inv_freq's 24-bit significand times 2^64 / 2 pi, shifted, is off by less than
// (|inv_freq| / 2 + 1) 2^-64 turns, and the product with pos wraps modulo one turn by
// itself. So a position of millions loses next to nothing (in float32 the angle's error
// alone would be pos * 2^-24), and neither double precision nor a range reduction is
// needed. The angle is then rounded to float32 in half turns (2^-25 at most, near a whole
// half turn). Rotations are computed in float32 and rounded once.
//
// Bound by memory: every row is read and written once (32,768 tokens of 32 query and
// 8 KV heads of 128: 135 us, 6.0 TB/s, 88 % of a plain copy). A warp takes one token
// and 32 / (d / 16) rows at a time; a lane holds 16 dims (8 pairs) of a row as
// 16-byte vectors and computes its 8 angles once for all rows of the token. A decode
// step (64 tokens: 4.8 us) is latency: three dependent loads and a launch, so the first
// row and the frequencies are loaded while the token's place is looked up, and a
// token's rows are shared among CTAs.
//
// k_append_codes: the 32-bit sign-projection codes of the appended keys
// (HashAttention: Semantic Sparsity for Faster Inference, Sec. 4.1), from the
// keys as the cache holds them, with the sums of hash_attn_encode_keys in the
// same order, so both give the same bits: dims k = u mod 4 in sequence for u = 0 .. 3, then
// (a0 + a1) + (a2 + a3). Bound by shared memory: a lane's tile of 4 bits x 4 keys reads 8
// vectors of 4 dims (24 wavefronts a warp) for 64 products of a warp, 1.5 times what the
// products take; a larger tile's sums (4 each) do not fit the registers. 16,384 tokens x 8
// heads of 128: 40 us, 27 TFLOP/s of float32 products. It starts beside k_append (staging W
// and looking up the places) and waits for it before it reads the keys: 64 tokens cost
// 3.8 us more with codes than without.
#include "ha_internal.cuh"

namespace ha {
namespace {

constexpr int kAppWarps = 4;   // (32,768 tokens of 32 + 8 heads of 128: 138 us with 8, 135 with 4)
constexpr int kCodeWarps = 8;

// inv_freq / 2 pi as a fraction of a turn in units of 2^-64 (finite inv_freq;
// whole turns drop out). 0x28BE60DB9391054A = floor(2^64 / 2 pi).
__device__ __forceinline__ unsigned long long turn_step(float f) {
    const uint32_t u = __float_as_uint(f);
    const int e = (int)((u >> 23) & 255u);
    const uint32_t sig = e != 0 ? ((u & 0x7fffffu) | 0x800000u) : (u & 0x7fffffu) << 1;
    const unsigned long long c = 0x28BE60DB9391054Aull;
    const unsigned long long hi = __umul64hi(c, sig), lo = c * sig;  // f = sig 2^(e - 150)
    const int s = 150 - e;
    unsigned long long r;
    if (s <= 0) r = s > -64 ? lo << -s : 0ull;
    else if (s < 64) r = (lo >> s) | (hi << (64 - s));
    else r = s < 128 ? hi >> (s - 64) : 0ull;
    return (u >> 31) ? 0ull - r : r;
}

// cos and sin of pos * step turns
__device__ __forceinline__ void turn(unsigned long long step, int pos, float& c, float& s) {
    const unsigned long long a = step * (unsigned long long)pos + 0x80000000ull;
    sincospif((float)(int32_t)(a >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
}

// Where the token of packed row t goes: its sequence s (cu[s] <= t < cu[s + 1]), and its
// position, or pos = -1 (skipped).
struct TokenPlace {
    int s, pos;
};
// True if sequence s owns row t; then x says where it goes. Three loads at once.
__device__ __forceinline__ bool owns(const AppendParams& p, int s, int t, TokenPlace& x) {
    const int a = p.cu[s], b = p.cu[s + 1], nk = p.seq_lens[s];
    if (a < 0 || a > t || t >= b) return false;
    x.s = s;
    x.pos = b > p.total || nk < 0 || nk > p.max_len ? -1 : max(-1, nk - (b - t));
    return true;
}
__device__ __forceinline__ TokenPlace place_of(const AppendParams& p, int t) {
    TokenPlace x{0, -1};
    // The sequences of a decode step, and prompts of one length, lie where an even split
    // has them: one look instead of a search (with the rows on their way meanwhile, 64
    // sequences of one token, 32 + 8 heads of 128: 5.6 -> 4.8 us).
    if (owns(p, min(p.n_seq - 1, (int)(((float)t + 0.5f) * p.seqs_per_row)), t, x)) return x;
    int lo = 0, hi = p.n_seq - 1;  // the last s with cu[s] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    owns(p, lo, t, x);
    return x;
}

template <typename T>
struct Vec8;  // 8 consecutive values
template <>
struct Vec8<__nv_bfloat16> {
    static __device__ __forceinline__ void load(const void* base, int64_t off, float (&x)[8]) {
        const uint4 w = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(base) + off);
        x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
        x[4] = bf16lo(w.z), x[5] = bf16hi(w.z), x[6] = bf16lo(w.w), x[7] = bf16hi(w.w);
    }
    static __device__ __forceinline__ void store(void* base, int64_t off, const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(base) + off) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec8<float> {
    static __device__ __forceinline__ void load(const void* base, int64_t off, float (&x)[8]) {
        const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + off);
        const float4 a = f[0], b = f[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    static __device__ __forceinline__ void store(void* base, int64_t off, const float (&x)[8]) {
        float4* f = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + off);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};

template <typename TI, typename TC, bool AXES>
__global__ void __launch_bounds__(kAppWarps * 32) k_append(const AppendParams p) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    // The kernel that writes the codes may read everything but the cache ahead of its wait. Any other
    // kernel of the library waits before it reads what an append may write.
    pdl_launch_dependents();
    if (blockIdx.y == 0 && p.flags != nullptr) {
        // the sequences' bounds, once
        for (int s = blockIdx.x * kAppWarps * 32 + tid; s < p.n_seq; s += gridDim.x * kAppWarps * 32) {
            const int a = p.cu[s], b = p.cu[s + 1], nk = p.seq_lens[s];
            if (a < 0 || b < a || b > p.total || nk < 0 || nk > p.max_len) atomicOr(p.flags, HA_DEVERR_SEQLEN);
            else if (nk < b - a) atomicOr(p.flags, HA_DEVERR_INDEX);
        }
    }
    const int t = blockIdx.x * kAppWarps + warp;
    if (t >= p.total) return;
    const int lanes = p.d >> 4, sub = lane / lanes, i = lane - sub * lanes, per = 32 / lanes;
    // this lane's two vectors of a rotated row, and its angles
    const bool turns = p.inv_freq != nullptr && 16 * i < p.rot;
    const int v0 = turns && !p.inter ? 8 * i : 16 * i;
    const int v1 = turns && !p.inter ? (p.rot >> 1) + 8 * i : 16 * i + 8;
    const int nq = p.q != nullptr ? p.Hq : 0, rows = nq + 2 * p.Hkv, step = gridDim.y * per;
    // row r of the token: 0 a query's, 1 a key's, 2 a value's; the head
    auto kind_of = [&](int r, int& h) {
        const int kind = r < nq ? 0 : (r < nq + p.Hkv ? 1 : 2);
        h = kind == 0 ? r : (kind == 1 ? r - nq : r - nq - p.Hkv);
        return kind;
    };
    auto load = [&](int r, float (&x)[8], float (&y)[8]) {
        int h;
        const int kind = kind_of(r, h);
        const void* src = kind == 0 ? p.q : (kind == 1 ? p.k : p.v);
        const int64_t st = kind == 0 ? p.q_st : (kind == 1 ? p.k_st : p.v_st), sh = kind == 0 ? p.q_sh : (kind == 1 ? p.k_sh : p.v_sh);
        const int64_t so = (int64_t)t * st + (int64_t)h * sh;
        Vec8<TI>::load(src, so + (kind == 2 ? 16 * i : v0), x);
        Vec8<TI>::load(src, so + (kind == 2 ? 16 * i + 8 : v1), y);
    };
    // the first row is on its way while the place is looked up, and the frequencies
    int r = blockIdx.y * per + sub;
    float x[8], y[8], f[8];
    if (r < rows) load(r, x, y);
    if (turns) {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = p.inv_freq[8 * i + k];
    }
    // the token's position on axis `lane`
    const int on_axis = AXES && lane < p.n_axes ? p.positions[lane * p.pos_st + t] : 0;
    const TokenPlace at = place_of(p, t);
    if (at.pos < 0) return;
    const int entry = at.pos / p.page_size, prow = at.pos - entry * p.page_size;
    const int page = p.table[(int64_t)at.s * p.table_st + entry];
    const bool good = page >= 0 && page < p.n_pages;
    if (!good && lane == 0 && p.flags != nullptr) atomicOr(p.flags, HA_DEVERR_INDEX);
    float c[8], sn[8];
    if constexpr (AXES) {
        const uint32_t axes = p.axes[i];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int pos = __shfl_sync(0xffffffffu, on_axis, (int)(axes >> (4 * k) & 15u));
            if (turns) turn(turn_step(f[k]), pos, c[k], sn[k]);
        }
    } else if (turns) {
#pragma unroll
        for (int k = 0; k < 8; ++k) turn(turn_step(f[k]), at.pos, c[k], sn[k]);
    }
    for (; r < rows; r += step) {
        if (r >= step) load(r, x, y);
        int h;
        const int kind = kind_of(r, h);
        const int a0 = kind == 2 ? 16 * i : v0, a1 = kind == 2 ? 16 * i + 8 : v1;
        if (turns && kind != 2) {
            if (p.inter) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float a = x[2 * k], b = x[2 * k + 1];
                    x[2 * k] = fmaf(a, c[k], -b * sn[k]);
                    x[2 * k + 1] = fmaf(b, c[k], a * sn[k]);
                    const float e = y[2 * k], f = y[2 * k + 1];
                    y[2 * k] = fmaf(e, c[4 + k], -f * sn[4 + k]);
                    y[2 * k + 1] = fmaf(f, c[4 + k], e * sn[4 + k]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float a = x[k], b = y[k];
                    x[k] = fmaf(a, c[k], -b * sn[k]);
                    y[k] = fmaf(b, c[k], a * sn[k]);
                }
            }
        }
        if (kind == 0) {
            const int64_t o = ((int64_t)t * p.Hq + h) * p.d;
            Vec8<TI>::store(p.q_out, o + a0, x);
            Vec8<TI>::store(p.q_out, o + a1, y);
        } else if (good) {
            char* dst = kind == 1 ? p.K : p.V;
            const int64_t o = kind == 1 ? (int64_t)page * p.k_sp + (int64_t)h * p.k_sc + (int64_t)prow * p.k_sn
                                        : (int64_t)page * p.v_sp + (int64_t)h * p.v_sc + (int64_t)prow * p.v_sn;
            Vec8<TC>::store(dst, o + a0, x);
            Vec8<TC>::store(dst, o + a1, y);
        }
    }
}

__device__ __forceinline__ void fma2(float2& acc, float a0, float a1, float b0, float b1) {
    uint64_t a, b, c;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
    asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(acc.x), "f"(acc.y));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(acc.x), "=f"(acc.y) : "l"(c));
}

// Lane (k, c) of a warp computes codes' bits c, c + 8, c + 16, c + 24 of the keys k, k + 4, ...
// (KPL of them).
template <typename TC, int D, int KPL>
__global__ void __launch_bounds__(kCodeWarps * 32, 2) k_append_codes(const AppendParams p) {
    constexpr int N = 4 * KPL;  // keys of a warp
    extern __shared__ __align__(16) float s_code[];  // W[g] [32][d + 4], then [kCodeWarps][N][d + 4] keys
    const int g = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int ld = D + 4, vecs = D / 8;  // rows 4 banks apart
    const float* Wg = p.W + (int64_t)g * 32 * D;
#pragma unroll
    for (int i = 0; i < 32 * D; i += kCodeWarps * 32) s_code[(i + tid) / D * ld + (i + tid) % D] = Wg[i + tid];
    float* xs = s_code + (32 + warp * N) * ld;
    const int kg = lane >> 3, cg = lane & 7;
    const float* wl = s_code + cg * ld;
    const float* xl = xs + kg * ld;
    bool first = true;
    for (int b0 = blockIdx.x * kCodeWarps * N; b0 < p.total; b0 += gridDim.x * kCodeWarps * N) {
        const int t0 = b0 + warp * N;
        int page = -1, row = 0;  // of this lane's key
        if (lane < N && t0 + lane < p.total) {
            const TokenPlace at = place_of(p, t0 + lane);
            if (at.pos >= 0) {
                const int e = at.pos / p.page_size;
                row = at.pos - e * p.page_size;
                page = p.table[(int64_t)at.s * p.table_st + e];
                if (page >= p.n_pages) page = -1;
            }
        }
        if (first) {
            pdl_wait();  // the keys are in the cache
            __syncthreads();
        }
        first = false;
#pragma unroll
        for (int i0 = 0; i0 < N * vecs; i0 += 32) {
            const int i = i0 + lane, v = i / vecs, e = i - v * vecs;
            const int pg = __shfl_sync(0xffffffffu, page, v), rw = __shfl_sync(0xffffffffu, row, v);
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (pg >= 0) Vec8<TC>::load(p.K, (int64_t)pg * p.k_sp + (int64_t)g * p.k_sc + (int64_t)rw * p.k_sn + 8 * e, x);
            float4* dst = reinterpret_cast<float4*>(xs + v * ld + 8 * e);
            dst[0] = make_float4(x[0], x[1], x[2], x[3]);
            dst[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
        __syncwarp();
        float2 lo[4][KPL], hi[4][KPL];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int q = 0; q < KPL; ++q) lo[c][q] = hi[c][q] = make_float2(0.f, 0.f);
#pragma unroll 2
        for (int k = 0; k < D; k += 4) {
            float4 w[4], x[KPL];
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const float4*>(wl + 8 * c * ld + k);
#pragma unroll
            for (int q = 0; q < KPL; ++q) x[q] = *reinterpret_cast<const float4*>(xl + 4 * q * ld + k);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int q = 0; q < KPL; ++q) {
                    fma2(lo[c][q], w[c].x, w[c].y, x[q].x, x[q].y);
                    fma2(hi[c][q], w[c].z, w[c].w, x[q].z, x[q].w);
                }
        }
        // a ballot gives byte k the bits c of key k
        uint32_t mine = 0;  // the code of key kg + 4 cg
#pragma unroll
        for (int q = 0; q < KPL; ++q) {
            uint32_t code = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float proj = (lo[c][q].x + lo[c][q].y) + (hi[c][q].x + hi[c][q].y);
                code |= ((__ballot_sync(0xffffffffu, proj > 0.f) >> (8 * kg)) & 255u) << (8 * c);
            }
            if (cg == q) mine = code;
        }
        const int key = kg + 4 * (cg & (KPL - 1));
        const int pg = __shfl_sync(0xffffffffu, page, key), rw = __shfl_sync(0xffffffffu, row, key);
        if (cg < KPL && pg >= 0) p.codes[(int64_t)pg * p.c_sp + (int64_t)g * p.c_sh + rw] = mine;
        __syncwarp();
    }
}

template <typename TC, int D, int KPL>
cudaError_t launch_codes(const AppendParams& p, cudaStream_t st) {
    const size_t smem = (size_t)(32 + kCodeWarps * 4 * KPL) * (D + 4) * sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(k_append_codes<TC, D, KPL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int per = kCodeWarps * 4 * KPL, blocks = (p.total + per - 1) / per;
    const int most = (2 * kSMs + p.Hkv - 1) / p.Hkv;  // two CTAs per SM in all: W is staged that often
    return launch_ex(k_append_codes<TC, D, KPL>, dim3((unsigned)(blocks < most ? blocks : most), (unsigned)p.Hkv),
                     dim3(kCodeWarps * 32), smem, st, true, p);
}

template <typename TI, typename TC>
cudaError_t launch_append_t(const AppendParams& p, cudaStream_t st) {
    const dim3 grid((unsigned)((p.total + kAppWarps - 1) / kAppWarps), (unsigned)p.row_splits);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kAppWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.W != nullptr && p.total < 2048) {
        // The codes' CTAs may start beside this kernel's only where its SM is set up for
        // shared memory already. 256 tokens x 8 heads: 11.2 -> 6.6 us, 1024: 14.5 -> 10.7;
        // 2048: 15.5 either way; 16,384: 58.5 -> 59.7, the copy itself misses the cache.
        attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
        attr[1].val.sharedMemCarveout = cudaSharedmemCarveoutMaxShared;
        cfg.numAttrs = 2;
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, p.positions != nullptr ? k_append<TI, TC, true> : k_append<TI, TC, false>, p);
    if (e != cudaSuccess || p.W == nullptr) return e;
    // Few keys: one a lane, as long as there is an SM for each CTA of 32 of them.
    // d 128, 8 heads, one key a lane / four: 64 tokens 6.4 / 8.7 us, 256: 6.6 / 10.1, 1024: 12.3 / 10.8.
    const bool few = (int64_t)p.total * p.Hkv < 32 * kSMs;
    if (p.d == 64) return few ? launch_codes<TC, 64, 1>(p, st) : launch_codes<TC, 64, 4>(p, st);
    return few ? launch_codes<TC, 128, 1>(p, st) : launch_codes<TC, 128, 4>(p, st);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p0, bool in_bf16, bool cache_bf16, cudaStream_t st) {
    AppendParams p = p0;
    p.seqs_per_row = (float)p.n_seq / (float)p.total;
    // a token's rows are shared among CTAs until there are about 16 warps per SM (64 tokens of
    // 48 rows: 4.8 us; a warp to a token: 8.5)
    const int per = 32 / (p.d >> 4), rows = (p.q != nullptr ? p.Hq : 0) + 2 * p.Hkv;
    const int steps = (rows + per - 1) / per, want = (16 * kSMs + p.total - 1) / p.total;
    p.row_splits = steps < want ? steps : want;
    if (in_bf16) return cache_bf16 ? launch_append_t<__nv_bfloat16, __nv_bfloat16>(p, st) : launch_append_t<__nv_bfloat16, float>(p, st);
    return cache_bf16 ? launch_append_t<float, __nv_bfloat16>(p, st) : launch_append_t<float, float>(p, st);
}

}  // namespace ha
