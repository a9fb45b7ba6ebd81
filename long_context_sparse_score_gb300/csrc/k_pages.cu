// The page plan of a serving step: page tables, row bounds, lengths and slots from the
// sequences' new lengths.
//
// Sequence s has had_s tokens in pages 0 .. p0 - 1 of its table row, p0 = ceil(had_s / ps), and
// gets nq_s more, in pages up to p1 = ceil((had_s + nq_s) / ps). Everything else is prefix sums over
// the sequences: rows cu_s = sum nq, places tb_s = sum (p1 - p0) among the pages taken, places fb_s
// = sum (pages given back). The free pages are a stack: an ended sequence's pages go to
// free[n_free + fb_s ..), page j of s is free[top - 1 - (tb_s + j - p0)] with top = n_free + all pages
// given back. So nothing waits for another sequence, and the result does not depend on timing.
//
// Bound by latency: a launch, the lengths, a scan, the pages, the table (64 sequences of one token,
// and 3,000 with 75,000 rows: see the measurements below). One cluster of up to 8 CTAs and no workspace:
// up to 1,024 sequences every CTA scans all of them, one to a thread, and they share the rows; more
// are cut among the CTAs, which tell each other their sums through distributed shared memory.
#include <cooperative_groups.h>

#include "ha_internal.cuh"

namespace cg = cooperative_groups;

namespace ha {
namespace {

constexpr int kMostThreads = 1024, kCluster = 8;
constexpr int kUnit = 256;    // rows that a warp writes at a time
constexpr int kDirect = 8;    // rows of a sequence that its own thread writes

struct PagesRecord {  // what the warps need of a sequence with many rows
    int row0, nq, had, tb, unit0;  // had -1: it is stopped
};

struct Sums {
    long long rows;
    uint32_t takes, back;
};

__device__ __forceinline__ uint32_t warp_incl(uint32_t x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += v;
    }
    return x;
}

__global__ void __launch_bounds__(kMostThreads) k_plan_pages(const PagesParams p) {
    __shared__ PagesRecord s_rec[kMostThreads];
    __shared__ uint32_t s_warp[4][32];
    __shared__ Sums s_sums, s_warp_sums[32];
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    pdl_wait();
    pdl_launch_dependents();

    // this CTA's sequences: all (then the rows are shared), or a part
    const bool all = p.n_seq <= (int)blockDim.x;
    const int per = all ? p.n_seq : (p.n_seq + C - 1) / C;
    const int s_begin = all ? 0 : min(p.n_seq, rank * per), s_end = min(p.n_seq, s_begin + per);
    const int n_tiles = max(1, (s_end - s_begin + (int)blockDim.x - 1) / (int)blockDim.x);
    const int max_len = p.max_pages * p.page_size;

    uint32_t flags = 0;
    int n_free = *p.n_free;
    if (n_free < 0 || n_free > p.n_pages) {
        flags |= HA_DEVERR_STATE;
        n_free = n_free < 0 ? 0 : p.n_pages;
    }

    // Sequence of this thread in a tile. state 0: none; 1: it goes on; 2: it ends; 3: it is stopped
    struct Mine {
        int s, had, nq, p0, state;
        uint32_t takes, back;
    } x;
    // Walks the entries of the warp's ended sequences, 32 at a time; put(place, page) for each that is a page.
    auto walk = [&](auto&& put) {
        uint32_t ended = __ballot_sync(0xffffffffu, x.state == 2 && x.p0 > 0);
        while (ended != 0) {
            const int l = __ffs((int)ended) - 1;
            ended &= ended - 1;
            const int pages = __shfl_sync(0xffffffffu, x.p0, l);
            const int32_t* row = p.table + (int64_t)__shfl_sync(0xffffffffu, x.s, l) * p.table_st;
            uint32_t n = 0;
            for (int j = lane; j - lane < pages; j += 32) {
                const int page = j < pages ? row[j] : -1;
                const uint32_t m = __ballot_sync(0xffffffffu, page >= 0 && page < p.n_pages);
                if (j < pages && (page < 0 || page >= p.n_pages)) flags |= HA_DEVERR_INDEX;
                put(l, n + (uint32_t)__popc((int)(m & ((1u << lane) - 1u))), page, (m >> lane) & 1u);
                n += (uint32_t)__popc((int)m);
            }
            if (lane == l) x.back = n;
        }
    };
    auto look = [&](int tile) {
        const int s = s_begin + tile * (int)blockDim.x + tid;
        x = Mine{s, 0, 0, 0, 0, 0u, 0u};
        if (s < s_end) {
            x.had = p.seq_lens[s];
            const int fresh = p.new_lens[s];
            const int tokens = min(x.had < 0 ? ~x.had : x.had, max_len);
            x.p0 = tokens / p.page_size + (tokens % p.page_size != 0 ? 1 : 0);
            x.nq = max(fresh, 0);
            if (fresh < 0) {
                x.state = 2;
            } else if (x.had < 0 || x.had > max_len || x.nq > max_len - x.had) {
                x.state = 3;
                if (x.had >= 0 || x.nq > 0) flags |= HA_DEVERR_SEQLEN;
            } else {
                x.state = 1;
                const int t = x.had + x.nq;
                x.takes = (uint32_t)(t / p.page_size + (t % p.page_size != 0 ? 1 : 0) - x.p0);
            }
        }
        walk([](int, uint32_t, int, uint32_t) {});
    };

    // ---- the sums, and those of the CTAs before
    Sums mine{0, 0u, 0u};
    for (int tile = 0; tile < n_tiles; ++tile) {
        look(tile);
        mine.rows += x.nq;
        mine.takes += x.takes;
        mine.back += x.back;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine.rows += __shfl_xor_sync(0xffffffffu, mine.rows, o);
    mine.takes = __reduce_add_sync(0xffffffffu, mine.takes);
    mine.back = __reduce_add_sync(0xffffffffu, mine.back);
    if (lane == 0) s_warp_sums[warp] = mine;
    __syncthreads();
    if (tid == 0) {
        Sums sum{0, 0u, 0u};
        for (int w = 0; w < warps; ++w) {
            sum.rows += s_warp_sums[w].rows;
            sum.takes += s_warp_sums[w].takes;
            sum.back += s_warp_sums[w].back;
        }
        s_sums = sum;
    }
    cluster.sync();  // every input has been read, too: outputs may lie where inputs did
    Sums before{0, 0u, 0u}, total{0, 0u, 0u};
    if (all) {
        total = s_sums;
    } else {
        for (int r = 0; r < C; ++r) {
            const Sums v = *cluster.map_shared_rank(&s_sums, r);
            if (r < rank) {
                before.rows += v.rows;
                before.takes += v.takes;
                before.back += v.back;
            }
            total.rows += v.rows;
            total.takes += v.takes;
            total.back += v.back;
        }
    }
    const bool over = total.rows > p.total;  // then nothing is planned
    uint32_t top = over ? (uint32_t)n_free : (uint32_t)n_free + min(total.back, (uint32_t)p.n_pages);
    if (top > (uint32_t)p.n_pages) {  // a page given back twice
        flags |= HA_DEVERR_STATE;
        top = (uint32_t)p.n_pages;
    }
    if (over) flags |= HA_DEVERR_COUNT;
    // which of several CTAs writes what belongs to sequence s
    auto writes = [&](int s) { return !all || s % C == rank; };

    // exclusive sum over the CTA's threads; `at` moves on by the CTA's sum
    auto scan = [&](int slot, uint32_t v, uint32_t& at) {
        const uint32_t incl = warp_incl(v, lane);
        if (lane == 31) s_warp[slot][warp] = incl;
        __syncthreads();
        uint32_t w = lane < warps ? s_warp[slot][lane] : 0u;
        w = warp_incl(w, lane);
        const uint32_t base = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0u;
        const uint32_t r = at + base + incl - v;
        at += __shfl_sync(0xffffffffu, w, 31);
        return r;
    };

    // ---- pages that come back
    if (!over && total.back != 0) {
        uint32_t at = before.back;
        for (int tile = 0; tile < n_tiles; ++tile) {
            if (n_tiles > 1) look(tile);
            const uint32_t fb = scan(0, x.back, at);
            walk([&](int l, uint32_t k, int page, uint32_t good) {
                const uint32_t i = (uint32_t)n_free + __shfl_sync(0xffffffffu, fb, l) + k;
                const int s = __shfl_sync(0xffffffffu, x.s, l);
                if (good && i < (uint32_t)p.n_pages && writes(s)) p.free_pages[i] = page;
            });
            __syncthreads();
        }
    }
    cluster.sync();  // (nobody reads another CTA's sums any more, either)

    // ---- lengths, bounds, tables, slots
    uint32_t at_rows = over ? 0u : (uint32_t)before.rows, at_takes = before.takes;
    for (int tile = 0; tile < n_tiles; ++tile) {
        if (n_tiles > 1) look(tile);
        const uint32_t row0 = scan(1, over ? 0u : (uint32_t)x.nq, at_rows), tb = scan(2, x.takes, at_takes);
        if (over) x.nq = 0;
        const bool fits = x.takes == 0u || tb + x.takes <= top;
        const bool goes = x.state == 1 && fits;
        const bool units = x.nq > kDirect;
        uint32_t n_units = 0;
        const uint32_t unit0 = scan(3, units ? (uint32_t)(x.nq + kUnit - 1) / kUnit : 0u, n_units);
        s_rec[tid] = PagesRecord{(int)row0, x.nq, goes ? x.had : -1, (int)tb, (int)unit0};
        if (x.state != 0 && writes(x.s)) {
            p.cu[x.s] = (int)row0;
            if (x.s == p.n_seq - 1) p.cu[p.n_seq] = (int)row0 + x.nq;
            int len = x.had;  // of a stopped sequence, as it is
            if (!over) {
                if (x.state == 2) len = 0;
                else if (goes) len = x.had + x.nq;
                else if (x.had >= 0 && x.had <= max_len) len = ~x.had;
                if (x.state == 1 && !fits) {
                    flags |= HA_DEVERR_PAGES;
                    if (tb <= top) *p.n_free_out = (int)(top - tb);  // the first that does not fit
                }
            }
            p.lens_out[x.s] = len;
        }
        auto pop = [&](uint32_t k) {  // (below top, as the sequence fits)
            const int page = __ldcg(p.free_pages + (top - 1u - k));
            if (page >= 0 && page < p.n_pages) return page;
            flags |= HA_DEVERR_INDEX;
            return -1;
        };
        // few rows: by their sequence's thread
        if (x.state != 0 && !over && !units && x.nq > 0 && writes(x.s)) {
            int32_t* row = p.table + (int64_t)x.s * p.table_st;
            int pg = x.had / p.page_size, r = x.had - pg * p.page_size, page = -1;
            if (goes && r != 0) page = row[pg];
            for (int i = 0; i < x.nq; ++i) {
                if (goes && r == 0) row[pg] = page = pop(tb + (uint32_t)(pg - x.p0));
                if (p.slots != nullptr) p.slots[row0 + (uint32_t)i] = goes && page >= 0 && page < p.n_pages ? page * p.page_size + r : -1;
                if (++r == p.page_size) r = 0, ++pg;
            }
        }
        __syncthreads();
        // many: by the warps, kUnit rows at a time
        for (uint32_t u = (uint32_t)(all ? warp * C + rank : warp); u < n_units; u += (uint32_t)(all ? warps * C : warps)) {
            int lo = 0, hi = (int)blockDim.x - 1;  // the last record that begins at or before u: it has units
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if ((uint32_t)s_rec[mid].unit0 <= u) lo = mid;
                else hi = mid - 1;
            }
            const PagesRecord rec = s_rec[lo];
            const int i0 = (int)(u - (uint32_t)rec.unit0) * kUnit, i1 = min(i0 + kUnit, rec.nq);
            if (rec.had < 0) {
                if (p.slots != nullptr)
                    for (int i = i0 + lane; i < i1; i += 32) p.slots[rec.row0 + i] = -1;
                continue;
            }
            int32_t* row = p.table + (int64_t)(s_begin + tile * (int)blockDim.x + lo) * p.table_st;
            const int p0 = (rec.had + p.page_size - 1) / p.page_size;
            // pages that begin in these rows
            const int b0 = rec.had + i0, b1 = rec.had + i1;
            for (int j = (b0 + p.page_size - 1) / p.page_size + lane; (int64_t)j * p.page_size < b1; j += 32)
                row[j] = pop((uint32_t)(rec.tb + j - p0));
            if (p.slots == nullptr) continue;
#pragma unroll 4
            for (int i = i0 + lane; i < i1; i += 32) {
                const int pos = rec.had + i, pg = pos / p.page_size;
                const int page = pg >= p0 ? pop((uint32_t)(rec.tb + pg - p0)) : row[pg];
                p.slots[rec.row0 + i] = page >= 0 && page < p.n_pages ? page * p.page_size + (pos - pg * p.page_size) : -1;
            }
        }
        __syncthreads();
    }
    if (rank == 0 && tid == 0) {
        if (over) *p.n_free_out = n_free;
        else if (total.takes <= top) *p.n_free_out = (int)(top - total.takes);
    }
    if (p.slots != nullptr) {
        const int64_t rows = over ? 0 : total.rows;
        for (int64_t t = rows + rank * (int64_t)blockDim.x + tid; t < p.total; t += (int64_t)C * blockDim.x) p.slots[t] = -1;
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0 && flags != 0u) flag_error(p.flags, flags);
}

}  // namespace

cudaError_t launch_plan_pages(const PagesParams& p, cudaStream_t st) {
    // One CTA as long as its threads have a sequence and a few rows each, else a cluster.
    const bool one = p.n_seq <= kMostThreads && p.total <= 4096;
    int threads = kMostThreads;
    if (one) {
        const int want = p.n_seq > p.total / 8 ? p.n_seq : p.total / 8;
        threads = want <= 128 ? 128 : (want + 31) / 32 * 32;
        if (threads > kMostThreads) threads = kMostThreads;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(one ? 1u : (unsigned)kCluster);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cfg.gridDim.x;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_plan_pages, p);
}

}  // namespace ha
