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
// Bound by latency: a launch, the lengths, a scan, the pages, the table. 64 sequences of one token 2.8 us
// (one CTA), 6 prompts of 39,000 tokens 5.2, 3,000 sequences of which 10 % add 85,000 tokens and 5 %
// end 13.2 (4.4 where all decode); the bytes would take 0.1. One CTA for up to 1,024 sequences with few rows,
// else one cluster of 8, and no workspace: up to kShared sequences every CTA scans all of them, one to a
// thread, and they share the rows; more are cut among the CTAs, which write their sums into each
// other's shared memory (1,000 sequences, 10 % prompts, 5 % ending: 13.3 us scanned by all, 10.4 cut; read
// from there behind the barrier the sums took 1.4 us).
#include <cooperative_groups.h>

#include "ha_internal.cuh"

namespace cg = cooperative_groups;

namespace ha {
namespace {

constexpr int kMostThreads = 1024, kThreads = 768, kCluster = 8;
constexpr int kUnit = 256;    // least rows that a warp writes at a time (PagesParams::unit)
constexpr int kShared = 128;  // sequences that all CTAs of a cluster look at
constexpr int kDirect = 8;    // rows of a sequence that its own thread writes
// A sum of rows that stays here is more than any buffer holds.
constexpr uint32_t kManyRows = 1u << 26;

struct PagesRecord {  // what the warps need of a sequence with many rows
    int row0, nq, had, tb, unit0;  // had -1: it is stopped
};
struct Ended {  // an ended sequence: its table's row, its pages, its place among the pages given back
    int s, pages;
    uint32_t at;
};

// What is summed over the sequences: new rows (up to kManyRows), pages taken, pages given back, units.
struct Sums {
    uint32_t rows, takes, back, units;
    __device__ __forceinline__ void add(const Sums& o) {
        rows = min(rows + o.rows, kManyRows);
        takes += o.takes;
        back += o.back;
        units += o.units;
    }
};
__device__ __forceinline__ Sums from_lane(const Sums& x, int l) {
    return Sums{__shfl_sync(0xffffffffu, x.rows, l), __shfl_sync(0xffffffffu, x.takes, l), __shfl_sync(0xffffffffu, x.back, l),
                __shfl_sync(0xffffffffu, x.units, l)};
}
__device__ __forceinline__ Sums scan_warp(Sums x, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sums v{__shfl_up_sync(0xffffffffu, x.rows, o), __shfl_up_sync(0xffffffffu, x.takes, o),
                     __shfl_up_sync(0xffffffffu, x.back, o), __shfl_up_sync(0xffffffffu, x.units, o)};
        if (lane >= o) x.add(v);
    }
    return x;
}

__global__ void __launch_bounds__(kMostThreads) k_plan_pages(const PagesParams p) {
    __shared__ PagesRecord s_rec[kMostThreads];
    __shared__ Ended s_ended[kMostThreads];
    __shared__ uint32_t s_back[kMostThreads];  // by thread: pages its ended sequence gives back
    __shared__ Sums s_warp[32], s_all[kCluster];  // s_all: the CTAs' sums, which each writes into all
    __shared__ int s_n_ended;
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    // this CTA's sequences: all (then the rows are shared), or a part
    const bool all = C == 1 || p.n_seq <= kShared;
    if (tid == 0) s_n_ended = 0;
    if (!all) cluster.barrier_arrive();  // a CTA's shared memory may be written once it runs
    pdl_wait();
    pdl_launch_dependents();

    const int per = all ? p.n_seq : (p.n_seq + C - 1) / C;
    const int s_begin = all ? 0 : min(p.n_seq, rank * per), s_end = min(p.n_seq, s_begin + per);
    const int n_tiles = max(1, (s_end - s_begin + (int)blockDim.x - 1) / (int)blockDim.x);
    const int max_len = p.max_pages * p.page_size;

    uint32_t flags = 0;
    int n_free = *p.n_free;

    // Sequence of this thread in a tile. state 0: none; 1: it goes on; 2: it ends; 3: it is stopped
    struct Mine {
        int s, had, nq, p0, state;
        uint32_t takes, back;
    } x;
    auto pages_of = [&](int tokens) {
        const int n = p.per_page(tokens);
        return n + (n * p.page_size < tokens ? 1 : 0);
    };
    auto page_ok = [&](int page) { return page >= 0 && page < p.n_pages; };
    // Entries of an ended sequence, 8 a lane at a time; put(place, page) for each that is a page. Returns their number.
    auto walk = [&](const Ended& e, auto&& put) {
        const int32_t* row = p.table + (int64_t)e.s * p.table_st;
        uint32_t n = 0;
        for (int j0 = 0; j0 < e.pages; j0 += 256) {
            int page[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int j = j0 + 32 * u + lane;
                page[u] = j < e.pages ? row[j] : -1;
                if (j < e.pages && !page_ok(page[u])) flags |= HA_DEVERR_INDEX;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint32_t m = __ballot_sync(0xffffffffu, page_ok(page[u]));
                if ((m >> lane) & 1u) put(n + (uint32_t)__popc((int)(m & ((1u << lane) - 1u))), page[u]);
                n += (uint32_t)__popc((int)m);
            }
        }
        return n;
    };
    // The tile's sequences; those that end are listed, and all warps count their pages.
    int listed = -1;  // this thread's place in s_ended
    auto look = [&](int tile) {
        listed = -1;
        const int s = s_begin + tile * (int)blockDim.x + tid;
        x = Mine{s, 0, 0, 0, 0, 0u, 0u};
        if (s < s_end) {
            x.had = p.seq_lens[s];
            const int fresh = p.new_lens[s];
            x.p0 = pages_of(min(x.had < 0 ? ~x.had : x.had, max_len));
            x.nq = max(fresh, 0);
            if (fresh < 0) {
                x.state = 2;
            } else if (x.had < 0 || x.had > max_len || x.nq > max_len - x.had) {
                x.state = 3;
                if (x.had >= 0 || x.nq > 0) flags |= HA_DEVERR_SEQLEN;
            } else {
                x.state = 1;
                x.takes = (uint32_t)(pages_of(x.had + x.nq) - x.p0);
            }
        }
        if (!__syncthreads_or(x.state == 2 && x.p0 > 0)) return;
        int at = -1;
        if (x.state == 2 && x.p0 > 0) {
            at = atomicAdd(&s_n_ended, 1);  // (their order does not matter: each has its place)
            s_ended[at] = Ended{s, x.p0, 0u};
        }
        __syncthreads();
        for (int i = warp; i < s_n_ended; i += warps) {
            const uint32_t n = walk(s_ended[i], [](uint32_t, int) {});
            if (lane == 0) s_back[i] = n;
        }
        __syncthreads();
        if (at >= 0) x.back = s_back[at];
        listed = at;
    };
    auto sums_of = [&]() {
        return Sums{(uint32_t)min(x.nq, (int)kManyRows), x.takes, x.back, x.nq > kDirect ? (uint32_t)p.per_unit(x.nq - 1) + 1u : 0u};
    };
    // Exclusive sums over the CTA's threads; total: all of them.
    auto scan = [&](Sums& total) {
        const Sums own = sums_of(), incl = scan_warp(own, lane);
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        const Sums upto = scan_warp(lane < warps ? s_warp[lane] : Sums{0u, 0u, 0u, 0u}, lane);
        total = from_lane(upto, 31);
        Sums before = from_lane(upto, max(warp - 1, 0));
        if (warp == 0) before = Sums{0u, 0u, 0u, 0u};
        const Sums prev{__shfl_up_sync(0xffffffffu, incl.rows, 1), __shfl_up_sync(0xffffffffu, incl.takes, 1),
                        __shfl_up_sync(0xffffffffu, incl.back, 1), __shfl_up_sync(0xffffffffu, incl.units, 1)};
        if (lane > 0) before.add(prev);
        __syncthreads();  // s_warp is free again
        return before;
    };

    // ---- the sums, and those of the CTAs before
    Sums mine{0u, 0u, 0u, 0u}, mine_before{0u, 0u, 0u, 0u};
    for (int tile = 0; tile < n_tiles; ++tile) {
        if (tile > 0) {
            __syncthreads();
            if (tid == 0) s_n_ended = 0;
            __syncthreads();
        }
        look(tile);
        Sums t;
        mine_before = scan(t);
        mine.add(t);
    }
    if (!all) cluster.barrier_wait();
    if (!all && tid < C) *cluster.map_shared_rank(&s_all[rank], tid) = mine;
    if (C > 1) cluster.sync();  // every input has been read, too: outputs may lie where inputs did
    else __syncthreads();
    if (n_free < 0 || n_free > p.n_pages) {
        flags |= HA_DEVERR_STATE;
        n_free = n_free < 0 ? 0 : p.n_pages;
    }
    Sums before{0u, 0u, 0u, 0u}, total = mine;
    if (!all) {
        const Sums v = lane < C ? s_all[lane] : Sums{0u, 0u, 0u, 0u};
        const Sums incl = scan_warp(v, lane);
        total = from_lane(incl, 31);
        if (rank > 0) before = from_lane(incl, rank - 1);
    }
    const bool over = total.rows > (uint32_t)p.total;  // then nothing is planned
    uint32_t top = over ? (uint32_t)n_free : (uint32_t)n_free + min(total.back, (uint32_t)p.n_pages);
    if (top > (uint32_t)p.n_pages) {  // a page given back twice
        flags |= HA_DEVERR_STATE;
        top = (uint32_t)p.n_pages;
    }
    if (over) flags |= HA_DEVERR_COUNT;
    // which of several CTAs writes what belongs to sequence s
    auto writes = [&](int s) { return !all || s % C == rank; };
    auto reload = [&](int tile) {  // of several tiles
        __syncthreads();
        if (tid == 0) s_n_ended = 0;
        __syncthreads();
        look(tile);
        Sums t;
        mine_before = scan(t);
        return t;
    };

    // ---- pages that come back
    if (total.back != 0) {
        Sums at = before;
        for (int tile = 0; !over && tile < n_tiles; ++tile) {
            Sums t = mine;
            if (n_tiles > 1) t = reload(tile);
            if (listed >= 0) s_ended[listed].at = at.back + mine_before.back;
            __syncthreads();
            for (int i = warp; i < s_n_ended; i += warps) {
                const Ended e = s_ended[i];
                if (!writes(e.s)) continue;
                walk(e, [&](uint32_t k, int page) {
                    const uint32_t to = (uint32_t)n_free + e.at + k;
                    if (to < (uint32_t)p.n_pages) p.free_pages[to] = page;
                });
            }
            at.add(t);
        }
    }
    if (C > 1 && total.back != 0) cluster.sync();  // before a page that was given back is taken
    else __syncthreads();

    // ---- lengths, bounds, tables, slots
    auto pop = [&](uint32_t k) {  // (below top, as the sequence fits)
        const int page = __ldcg(p.free_pages + (top - 1u - k));
        if (page_ok(page)) return page;
        flags |= HA_DEVERR_INDEX;
        return -1;
    };
    Sums at = before;
    for (int tile = 0; tile < n_tiles; ++tile) {
        Sums t = mine;
        if (n_tiles > 1) t = reload(tile);
        const uint32_t row0 = over ? 0u : at.rows + mine_before.rows, tb = at.takes + mine_before.takes;
        if (over) x.nq = 0;
        const bool fits = x.takes == 0u || tb + x.takes <= top;
        const bool goes = x.state == 1 && fits;
        s_rec[tid] = PagesRecord{(int)row0, x.nq, goes ? x.had : -1, (int)tb, (int)mine_before.units};
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
            // few rows: by their sequence's thread
            if (x.nq > 0 && x.nq <= kDirect) {
                int32_t* row = p.table + (int64_t)x.s * p.table_st;
                int pg = p.per_page(max(x.had, 0)), r = x.had - pg * p.page_size, page = -1;
                if (goes && r != 0) page = row[pg];
                for (int i = 0; i < x.nq; ++i) {
                    if (goes && r == 0) row[pg] = page = pop(tb + (uint32_t)(pg - x.p0));
                    if (p.slots != nullptr) p.slots[row0 + (uint32_t)i] = goes && page_ok(page) ? page * p.page_size + r : -1;
                    if (++r == p.page_size) r = 0, ++pg;
                }
            }
        }
        __syncthreads();
        // many: by the warps, p.unit rows at a time (32 rows on are so many pages and rows on: the one
        // division of a row would be most of what it costs)
        const int step_pages = p.per_page(32), step_rows = 32 - step_pages * p.page_size;
        const uint32_t n_units = over ? 0u : t.units;
        for (uint32_t u = (uint32_t)(all ? warp * C + rank : warp); u < n_units; u += (uint32_t)(all ? warps * C : warps)) {
            // the last record that begins at or before u (it has units): of 32 groups of records, then of the group's
            int lo = 32 * lane < (int)blockDim.x && (uint32_t)s_rec[32 * lane].unit0 <= u ? 1 : 0;
            lo = 32 * (31 - __clz((int)__ballot_sync(0xffffffffu, lo != 0)));
            lo += 31 - __clz((int)__ballot_sync(0xffffffffu, (uint32_t)s_rec[lo + lane].unit0 <= u));
            const PagesRecord rec = s_rec[lo];
            const int i0 = (int)(u - (uint32_t)rec.unit0) * p.unit, i1 = min(i0 + p.unit, rec.nq);
            if (rec.had < 0) {
                if (p.slots != nullptr)
                    for (int i = i0 + lane; i < i1; i += 32) p.slots[rec.row0 + i] = -1;
                continue;
            }
            int32_t* row = p.table + (int64_t)(s_begin + tile * (int)blockDim.x + lo) * p.table_st;
            const int p0 = pages_of(rec.had), b0 = rec.had + i0, b1 = rec.had + i1;
            // 32 of the unit's pages at a time, one to a lane, and the rows in them
            const int pg1 = p.per_page(b1 - 1);
            for (int pg0 = p.per_page(b0); pg0 <= pg1; pg0 += 32) {
                const int pg = pg0 + lane;
                int page = -1;
                if (pg <= pg1) {
                    page = pg >= p0 ? pop((uint32_t)(rec.tb + pg - p0)) : row[pg];
                    if (pg >= p0 && (int64_t)pg * p.page_size >= b0) row[pg] = page;  // it begins here
                }
                if (p.slots == nullptr) continue;
                const int r0 = max(b0, pg0 * p.page_size);
                const int r1 = (int)min((int64_t)b1, ((int64_t)pg0 + 32) * p.page_size);
                int e = p.per_page(r0 + lane), off = r0 + lane - e * p.page_size;  // of this lane's row
#pragma unroll 4
                for (int q0 = r0; q0 < r1; q0 += 32) {
                    const int of = __shfl_sync(0xffffffffu, page, min(e - pg0, 31)), pos = q0 + lane;
                    if (pos < r1) p.slots[rec.row0 + (pos - rec.had)] = page_ok(of) ? of * p.page_size + off : -1;
                    e += step_pages;
                    off += step_rows;
                    if (off >= p.page_size) off -= p.page_size, ++e;
                }
            }
        }
        at.add(t);
    }
    if (rank == 0 && tid == 0) {
        if (over) *p.n_free_out = n_free;
        else if (total.takes <= top) *p.n_free_out = (int)(top - total.takes);
    }
    if (p.slots != nullptr) {
        const int rows = over ? 0 : (int)total.rows;
        for (int t = rows + rank * (int)blockDim.x + tid; t < p.total; t += C * (int)blockDim.x) p.slots[t] = -1;
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0 && flags != 0u) flag_error(p.flags, flags);
}

}  // namespace

cudaError_t launch_plan_pages(const PagesParams& p0, cudaStream_t st) {
    PagesParams p = p0;
    p.per_page = Quotient::of((uint32_t)p.page_size);
    // What a warp does once for its rows (the search, the pages) costs as much as 200 rows, so with many rows it
    // takes more of them (3,000 mixed sequences 16.6 -> 13.5 us, with pages found by a product instead of a division).
    p.unit = p.total / 128 > kUnit ? p.total / 128 : kUnit;
    p.per_unit = Quotient::of((uint32_t)p.unit);
    // One CTA as long as its threads have a sequence and a few rows each, else a cluster.
    const bool one = p.n_seq <= kMostThreads && p.total <= 4096;
    // 768 threads: a barrier of fewer warps, as long as each has a sequence (3,000 mixed sequences 13.4 -> 13.1 us, all
    // decoding 4.9 -> 4.4, 6 prompts 5.6 -> 5.2; with 512 14.6, 3.9 and 5.0).
    int threads = p.n_seq <= kCluster * kThreads ? kThreads : kMostThreads;
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
