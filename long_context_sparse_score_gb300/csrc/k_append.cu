// Append new tokens to a paged KV cache, rotating queries and keys by their
// positions on the way.
//
// k_append: token i of sequence s (nq new tokens, nk tokens once they are in)
// sits at position pos = nk - nq + i, in row pos % page_size of page
// table[s][pos / page_size]. Its queries and keys are rotated: pair p of the
// first `rot` dims, (x_p, x_{p + rot/2}) or, interleaved, (x_{2p}, x_{2p+1}),
// turns by the angle pos * inv_freq[p]; the other dims and the values are copied.
//
// The angle in turns, pos * inv_freq / 2 pi, is kept as a 64-bit fixed-point
// fraction: inv_freq's 24-bit significand times 2^64 / 2 pi, shifted, is exact to
// 2^-64 turns, and the product with pos wraps modulo one turn by itself. So a
// position of millions loses nothing (in float32 the angle's error alone would
// be pos * 2^-24), and neither double precision nor a range reduction is needed.
// Rotations are computed in float32 and rounded once.
//
// Bound by memory: every row is read and written once. A warp takes one token
// and 32 / (d / 16) rows at a time; a lane holds 16 dims (8 pairs) of a row as
// 16-byte vectors and computes its 8 angles once for all rows of the token.
//
// k_append_codes: the 32-bit sign-projection codes of the appended keys
// (HashAttention: Semantic Sparsity for Faster Inference, Sec. 4.1), from the
// keys as the cache holds them, with the sums of hash_attn_encode_keys in the
// same order, so both give the same bits. A CTA stages W[g] once; a warp runs 8
// keys at a time, so that a weight read from shared memory serves 8 products.
#include "ha_internal.cuh"

namespace ha {
namespace {

constexpr int kAppWarps = 8;
constexpr int kCodeKeys = 8;  // keys a warp projects at a time

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

// The sequence that owns packed row t (cu[s] <= t < cu[s + 1]), or -1; warp-wide,
// 32 boundaries a step.
__device__ __forceinline__ int find_seq(const int32_t* cu, int n_seq, int t, int lane) {
    int lo = 0, n = n_seq;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool le = lane * step < n && cu[i] <= t;
        const int k = 31 - __clz((int)(__ballot_sync(0xffffffffu, le) | 1u));
        lo += k * step;
        n = min(step, n - k * step);
    }
    return (cu[lo] >= 0 && cu[lo] <= t && t < cu[lo + 1]) ? lo : -1;
}

// Where the token of row t goes: its position, or -1 (skipped).
__device__ __forceinline__ int place_of(const AppendParams& p, int s, int t) {
    if (s < 0) return -1;
    const int a = p.cu[s], b = p.cu[s + 1], nk = p.seq_lens[s];
    if (b > p.total || nk < 0 || nk > p.max_len) return -1;
    const int pos = nk - (b - t);
    return pos < 0 || t < a ? -1 : pos;
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

template <typename TI, typename TC>
__global__ void __launch_bounds__(kAppWarps * 32) k_append(const AppendParams p) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && blockIdx.y == 0 && p.flags != nullptr) {
        // the sequences' bounds, once
        for (int s = tid; s < p.n_seq; s += kAppWarps * 32) {
            const int a = p.cu[s], b = p.cu[s + 1], nk = p.seq_lens[s];
            if (a < 0 || b < a || b > p.total || nk < 0 || nk > p.max_len) atomicOr(p.flags, HA_DEVERR_SEQLEN);
            else if (nk < b - a) atomicOr(p.flags, HA_DEVERR_INDEX);
        }
    }
    const int t = blockIdx.x * kAppWarps + warp;
    if (t >= p.total) return;
    const int s = find_seq(p.cu, p.n_seq, t, lane);
    const int pos = place_of(p, s, t);
    if (pos < 0) return;
    const int lanes = p.d >> 4, sub = lane / lanes, i = lane - sub * lanes, per = 32 / lanes;
    const int entry = pos / p.page_size, prow = pos - entry * p.page_size;
    const int page = p.table[(int64_t)s * p.table_st + entry];
    const bool good = page >= 0 && page < p.n_pages;
    if (!good && lane == 0 && p.flags != nullptr) atomicOr(p.flags, HA_DEVERR_INDEX);
    // this lane's two vectors of a rotated row, and its angles
    const bool turns = p.inv_freq != nullptr && 16 * i < p.rot;
    const int v0 = turns && !p.inter ? 8 * i : 16 * i;
    const int v1 = turns && !p.inter ? (p.rot >> 1) + 8 * i : 16 * i + 8;
    float c[8], sn[8];
    if (turns) {
#pragma unroll
        for (int k = 0; k < 8; ++k) turn(turn_step(p.inv_freq[8 * i + k]), pos, c[k], sn[k]);
    }
    const int nq = p.q != nullptr ? p.Hq : 0;
    const int rows = nq + 2 * p.Hkv;
    for (int r = blockIdx.y * per + sub; r < rows; r += gridDim.y * per) {
        const void* src;
        int64_t so;
        int kind = 0, h = r;  // query, key, value
        if (r < nq) {
            src = p.q;
            so = (int64_t)t * p.q_st + (int64_t)h * p.q_sh;
        } else if (r < nq + p.Hkv) {
            kind = 1;
            h = r - nq;
            src = p.k;
            so = (int64_t)t * p.k_st + (int64_t)h * p.k_sh;
        } else {
            kind = 2;
            h = r - nq - p.Hkv;
            src = p.v;
            so = (int64_t)t * p.v_st + (int64_t)h * p.v_sh;
        }
        const int a0 = kind == 2 ? 16 * i : v0, a1 = kind == 2 ? 16 * i + 8 : v1;
        float x[8], y[8];
        Vec8<TI>::load(src, so + a0, x);
        Vec8<TI>::load(src, so + a1, y);
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

template <typename TC>
__global__ void __launch_bounds__(kAppWarps * 32) k_append_codes(const AppendParams p) {
    extern __shared__ float s_code[];  // W[g] transposed [d][33], then [kAppWarps][kCodeKeys][d] keys
    const int g = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float* Wg = p.W + (int64_t)g * 32 * p.d;
    for (int i = tid; i < 32 * p.d; i += kAppWarps * 32) {
        const int j = i / p.d, k = i - j * p.d;
        s_code[k * 33 + j] = Wg[i];
    }
    __syncthreads();
    float* xs = s_code + ((p.d * 33 + 3) & ~3) + warp * kCodeKeys * p.d;
    for (int t0 = (blockIdx.x * kAppWarps + warp) * kCodeKeys; t0 < p.total; t0 += gridDim.x * kAppWarps * kCodeKeys) {
        int page[kCodeKeys], row[kCodeKeys];
#pragma unroll
        for (int v = 0; v < kCodeKeys; ++v) {
            const int t = t0 + v;
            page[v] = -1;
            row[v] = 0;
            if (t < p.total) {
                const int s = find_seq(p.cu, p.n_seq, t, lane);
                const int pos = place_of(p, s, t);
                if (pos >= 0) {
                    const int e = pos / p.page_size;
                    row[v] = pos - e * p.page_size;
                    page[v] = p.table[(int64_t)s * p.table_st + e];
                    if (page[v] >= p.n_pages) page[v] = -1;
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int v = 0; v < kCodeKeys; ++v) {
            for (int i = lane; i < p.d / 8; i += 32) {
                float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (page[v] >= 0)
                    Vec8<TC>::load(p.K, (int64_t)page[v] * p.k_sp + (int64_t)g * p.k_sc + (int64_t)row[v] * p.k_sn + 8 * i, x);
#pragma unroll
                for (int k = 0; k < 8; ++k) xs[v * p.d + 8 * i + k] = x[k];
            }
        }
        __syncwarp();
        float acc[kCodeKeys][4];
#pragma unroll
        for (int v = 0; v < kCodeKeys; ++v)
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[v][u] = 0.f;
        for (int k = 0; k < p.d; k += 4) {
            float w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) w[u] = s_code[(k + u) * 33 + lane];
#pragma unroll
            for (int v = 0; v < kCodeKeys; ++v) {
                const float4 x = *reinterpret_cast<const float4*>(xs + v * p.d + k);
                acc[v][0] = fmaf(w[0], x.x, acc[v][0]);
                acc[v][1] = fmaf(w[1], x.y, acc[v][1]);
                acc[v][2] = fmaf(w[2], x.z, acc[v][2]);
                acc[v][3] = fmaf(w[3], x.w, acc[v][3]);
            }
        }
#pragma unroll
        for (int v = 0; v < kCodeKeys; ++v) {
            const float proj = (acc[v][0] + acc[v][1]) + (acc[v][2] + acc[v][3]);
            const uint32_t code = __ballot_sync(0xffffffffu, proj > 0.f);
            if (lane == 0 && page[v] >= 0)
                p.codes[(int64_t)page[v] * p.c_sp + (int64_t)g * p.c_sh + row[v]] = code;
        }
        __syncwarp();
    }
}

template <typename TI, typename TC>
cudaError_t launch_append_t(const AppendParams& p, cudaStream_t st) {
    const dim3 grid((unsigned)((p.total + kAppWarps - 1) / kAppWarps), (unsigned)p.row_splits);
    k_append<TI, TC><<<grid, kAppWarps * 32, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.W == nullptr) return e;
    const size_t smem = (((size_t)p.d * 33 + 3) / 4 * 4 + (size_t)kAppWarps * kCodeKeys * p.d) * sizeof(float);
    e = cudaFuncSetAttribute(k_append_codes<TC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int per = kAppWarps * kCodeKeys, blocks = (p.total + per - 1) / per;
    const int most = (4 * kSMs + p.Hkv - 1) / p.Hkv;  // four CTAs per SM in all: W is staged that often
    k_append_codes<TC><<<dim3((unsigned)(blocks < most ? blocks : most), (unsigned)p.Hkv), kAppWarps * 32, smem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendParams& p0, bool in_bf16, bool cache_bf16, cudaStream_t st) {
    AppendParams p = p0;
    // a token's rows are shared among CTAs until there are about 16 warps per SM
    const int per = 32 / (p.d >> 4), rows = (p.q != nullptr ? p.Hq : 0) + 2 * p.Hkv;
    const int steps = (rows + per - 1) / per, want = (16 * kSMs + p.total - 1) / p.total;
    p.row_splits = steps < want ? steps : want;
    if (in_bf16) return cache_bf16 ? launch_append_t<__nv_bfloat16, __nv_bfloat16>(p, st) : launch_append_t<__nv_bfloat16, float>(p, st);
    return cache_bf16 ? launch_append_t<float, __nv_bfloat16>(p, st) : launch_append_t<float, float>(p, st);
}

}  // namespace ha
