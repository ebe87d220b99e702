// kv_evict.cuh -- eviction from a KV cache by accumulated attention weight.
//
// Per (entry, kv head): of the P rows, `keep` stay.  Rows at positions >= tokens - recent come first, then
// the rows by decreasing weight, ties to the lowest row (keep = 0: none, and nothing moves).  Kept rows below
// `keep` stay where they are; the i-th kept row at or past `keep` (a mover) goes to the i-th row below `keep`
// that is not kept (a hole), so a call moves no more rows than it must, and sources (at or past keep) and
// targets (below it) never overlap.  Attention over the prefix does not depend on the order of its rows; pos
// says which token each one is.
//
// One launch: a cluster of 1 to 8 blocks per (entry, kv head), each with a slice of the rows.  It reads 8 bytes a row
// once, keeps the slice's ranks in shared memory (up to 32768 rows), and finds the keep-th largest by 11, 11 and 10
// bits in turn, from histograms that the blocks read from each other (distributed shared memory); eleven bits tell
// weights apart that share an exponent, so few lanes meet in a bin, and a pass whose bin stays whole is the last.  Then
// every warp counts the holes and movers of its rows, and their places in the lists follow from the counts ahead of
// it: no sort, and no order that depends on timing.  The cluster's warps then move the rows, K and V, eight at a time.
// The new lengths may lie where the old ones do: the last cluster to have read its own writes them all.
//
// 256 heads of 2064 rows, 16 moves each: 10.9 us, bound by a dozen block-wide steps.  32 heads of 32768 rows to 8192 on
// clusters of four: 56 us, of which about 19 find the rows and 38 move 198 MB in rows of 256 bytes (5.2 TB/s); half
// the warps moving: 71 us.  Two launches, the second moving the rows from the whole GPU, took 14.8 and 62 us, 2 to 3 us
// more outside a graph, and were faster only where few heads leave SMs idle (8 heads of 32768 rows: 40.6 against 43.5).
// 64 registers, so that 512-thread blocks share an SM in pairs: 22 us for the 256 heads without.
#pragma once

#include <cstdint>

#include <cooperative_groups.h>

#include "evict_select.cuh"
#include "kv_paged.cuh"

namespace e2d2 {

constexpr int kEvictRows = 32768;  // rows whose ranks a block can hold in shared memory

struct EvictParams {
    PageView pages;
    uint4* pool[2];       // K, V pools
    const int* P_dev;
    const float* weight;  // [B][Hkv][capacity]
    const int* pos;
    const int* tokens;
    float* weight_out;    // the same arrays, or others
    int* pos_out;
    int* P_out;
    int* heads_done;      // zero between calls
    int* ws;              // per unit: list_rows holes, list_rows movers
    int batch, keep, recent;
    int list_rows;
    int rank_rows;        // rows that the launch's shared memory has ranks for
    long long ws_stride;
};

// Rank of a row, larger for rows that stay: unsigned integers in the order of the floats, -0 as 0, NaN below
// every number, protected rows above all.
__device__ __forceinline__ uint32_t evict_rank(float w, int pos, int protect_from) {
    if (pos >= protect_from) return 0xffffffffu;
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of x over the block's warps (x: the same in all lanes of a warp), *total their sum.
template <int WARPS>
__device__ __forceinline__ int warps_exclusive(int x, int* wsum, int* total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    __syncthreads();  // the previous call's sums have been read
    if (lane == 0) wsum[wid] = x;
    __syncthreads();
    const int mine = lane < WARPS ? wsum[lane] : 0;
    *total = __reduce_add_sync(0xffffffffu, mine);
    return __reduce_add_sync(0xffffffffu, lane < wid ? mine : 0);
}

// VPR: 16-byte vectors per row of K or V.
template <int THREADS, int VPR>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) kv_evict_kernel(const __grid_constant__ EvictParams p) {
    namespace cg = cooperative_groups;
    constexpr int WARPS = THREADS / 32, BINS = kEvictBins / THREADS, BATCH = 8;
    __shared__ __align__(16) unsigned int hist[2][kEvictBins];
    __shared__ int wsum[WARPS];
    __shared__ EvictPick s_pick;
    __shared__ int s_count[3];          // this block's rows at the threshold, holes, movers
    extern __shared__ uint32_t ranks[]; // [rank_rows]
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = static_cast<int>(cluster.num_blocks()), me = static_cast<int>(cluster.block_rank());
    // every thread of the cluster; a cluster's barrier costs half a microsecond more than a block's (256 heads of 2064 rows on
    // one block each: 13.0 against 10.9 us)
    auto meet = [&]() {
        if (blocks == 1) __syncthreads();
        else cluster.sync();
    };
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    for (int i = tid; i < 2 * kEvictBins; i += THREADS) (&hist[0][0])[i] = 0;
    ptx::griddep_wait();
    const int unit = blockIdx.x / blocks, Hkv = p.pages.kv_heads, cap = p.pages.capacity();
    const int b = unit / Hkv, h = unit - b * Hkv;
    const int P = ragged_clamp(__ldcg(p.P_dev + b), cap);
    // the first protected position, without overflow for any recent >= 0
    const long long pf = static_cast<long long>(__ldcg(p.tokens + b)) - p.recent;
    const int protect = pf < INT_MIN ? INT_MIN : static_cast<int>(pf);
    const long long row0 = static_cast<long long>(unit) * cap;
    const float* w = p.weight + row0;
    const int* pos = p.pos + row0;
    float* w_out = p.weight_out + row0;
    int* pos_out = p.pos_out + row0;
    int* ws = p.ws + unit * p.ws_stride;
    const bool copy = w_out != w || pos_out != pos;
    const int per = ((P + blocks - 1) / blocks + 31) / 32 * 32;  // rows of a block
    const int beg = min(me * per, P), rows = min(beg + per, P) - beg;
    // By one warp, when all of the cluster has read the length.
    auto head_done = [&]() {
        int before = 0;
        if (lane == 0) {
            __threadfence();
            before = atomicAdd(p.heads_done, 1);
        }
        if (__shfl_sync(0xffffffffu, before, 0) != p.batch * Hkv - 1) return;
        __threadfence();
        for (int e = lane; e < p.batch; e += 32) p.P_out[e] = min(ragged_clamp(__ldcg(p.P_dev + e), cap), p.keep);
        if (lane == 0) *p.heads_done = 0;
    };
    // The same for every block of the cluster: one that reads the length after head_done() has let it be written finds
    // min(P, keep), for which this holds too.
    if (!evict_selects(P, p.keep)) {
        if (copy)
            for (int j = beg + tid; j < min(beg + rows, p.keep); j += THREADS) {
                w_out[j] = __ldcg(w + j);
                pos_out[j] = __ldcg(pos + j);
            }
        if (me == blocks - 1 && wid == WARPS / 2) head_done();
        return;
    }
    const bool held = rows <= p.rank_rows;
    auto rank_of = [&](int i) { return held ? ranks[i] : evict_rank(__ldcg(w + beg + i), __ldcg(pos + beg + i), protect); };
    __syncthreads();

    // One read of the rows: their ranks, the first histogram, and (unless in place) the copy of the rows below keep;
    // the movers overwrite the holes among them at the end.
#pragma unroll 1
    for (int i0 = tid; i0 < rows; i0 += BATCH * THREADS) {
        float wv[BATCH];
        int pv[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = i0 + k * THREADS;
            if (i < rows) wv[k] = __ldcg(w + beg + i), pv[k] = __ldcg(pos + beg + i);
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = i0 + k * THREADS;
            if (i >= rows) break;
            const uint32_t r = evict_rank(wv[k], pv[k], protect);
            if (held) ranks[i] = r;
            atomicAdd(&hist[0][r >> 21], 1u);
            if (copy && beg + i < p.keep) w_out[beg + i] = wv[k], pos_out[beg + i] = pv[k];
        }
    }
    // The keep-th largest rank, 11, 11 and 10 bits a pass: prefix = its leading bits, need = how many rows with that
    // prefix stay; done when all of them do.
    unsigned int prefix = 0, need = p.keep, equal = 0;
    int shift = evict_pass_shift(0), bits = evict_pass_bits(0);
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        if (pass > 0) {
            const unsigned int mask = (1u << bits) - 1u;
#pragma unroll 4
            for (int i = tid; i < rows; i += THREADS) {
                const uint32_t r = rank_of(i);
                if ((r >> (shift + bits)) == prefix) atomicAdd(&hist[pass & 1][(r >> shift) & mask], 1u);
            }
        }
        meet();
        // bins from the largest down, BINS of them per thread: the one where the count from above reaches need
        unsigned int mine[BINS], sum = 0;
#pragma unroll
        for (int i = 0; i < BINS; ++i) mine[i] = 0;
        for (int c = 0; c < blocks; ++c) {
            const unsigned int* h = cluster.map_shared_rank(&hist[pass & 1][0], c) + kEvictBins - BINS * (tid + 1);
            if constexpr (BINS % 4 == 0) {
#pragma unroll
                for (int i = 0; i < BINS; i += 4) {
                    const uint4 x = *reinterpret_cast<const uint4*>(h + BINS - 4 - i);
                    mine[i] += x.w, mine[i + 1] += x.z, mine[i + 2] += x.y, mine[i + 3] += x.x;
                }
            } else {
#pragma unroll
                for (int i = 0; i < BINS; ++i) mine[i] += h[BINS - 1 - i];
            }
        }
#pragma unroll
        for (int i = 0; i < BINS; ++i) sum += mine[i];
        unsigned int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned int y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        int all;
        unsigned int above = warps_exclusive<WARPS>(static_cast<int>(__shfl_sync(0xffffffffu, inc, 31)), wsum, &all) + inc - sum;
        // every block has read the other histogram (the cluster has met since): it is clear for the pass after next
        if (pass == 1)
            for (int i = tid; i < kEvictBins; i += THREADS) hist[0][i] = 0;
        EvictPick next;
        if (evict_pick<BINS>(mine, above, sum, need, tid, bits, prefix, next)) s_pick = next;
        __syncthreads();
        prefix = s_pick.prefix;
        need = s_pick.need;
        equal = s_pick.equal;
        if (need == equal || shift == 0) break;
        bits = evict_pass_bits(pass + 1);
        shift = evict_pass_shift(pass + 1);
    }
    // Rows above the threshold stay, and the first `need` of the `equal` rows at it.  A warp takes a run of the
    // block's rows, 32 at a time, in their order.
    int* hole_list = ws;
    int* mover_list = hole_list + p.list_rows;
    const int run = ((rows + WARPS - 1) / WARPS + 31) / 32 * 32;
    const int i_beg = min(wid * run, rows), i_end = min(i_beg + run, rows);
    const bool ties = need != equal;
    int eq_before = 0;  // rows at the threshold ahead of this warp's
    if (ties) {
        int n = 0, all;
        for (int i = i_beg; i < i_end; i += 32)
            n += __popc(__ballot_sync(0xffffffffu, i + lane < rows && (rank_of(min(i + lane, rows - 1)) >> shift) == prefix));
        eq_before = warps_exclusive<WARPS>(n, wsum, &all);
        if (tid == 0) s_count[0] = all;
        meet();
        for (int c = 0; c < me; ++c) eq_before += *cluster.map_shared_rank(&s_count[0], c);
    }
    // whether row i stays; `eqs` counts the rows at the threshold on the way
    auto stays = [&](int i, int& eqs) {
        const uint32_t r = (i < rows ? rank_of(i) : 0u) >> shift;
        const bool eq = i < rows && r == prefix;
        bool stay = i < rows && r >= prefix;
        if (ties) {
            const uint32_t m = __ballot_sync(0xffffffffu, eq);
            if (eq) stay = eqs + __popc(m & ((1u << lane) - 1u)) < static_cast<int>(need);
            eqs += __popc(m);
        }
        return stay;
    };
    int holes = 0, movers = 0, eqs = eq_before;
#pragma unroll 4
    for (int i = i_beg; i < i_end; i += 32) {
        const bool stay = stays(i + lane, eqs), in = i + lane < rows, low = beg + i + lane < p.keep;
        holes += __popc(__ballot_sync(0xffffffffu, in && low && !stay));
        movers += __popc(__ballot_sync(0xffffffffu, in && !low && stay));
    }
    int all_holes, all_movers;
    holes = warps_exclusive<WARPS>(holes, wsum, &all_holes);
    movers = warps_exclusive<WARPS>(movers, wsum, &all_movers);
    if (tid == 0) {
        s_count[1] = all_holes;
        s_count[2] = all_movers;
    }
    meet();
    int moves = 0;
    for (int c = 0; c < blocks; ++c) {
        const int* n = cluster.map_shared_rank(&s_count[0], c);
        if (c < me) holes += n[1], movers += n[2];
        moves += n[2];
    }
    eqs = eq_before;
#pragma unroll 4
    for (int i = i_beg; i < i_end; i += 32) {
        const int j = beg + i + lane;
        const bool stay = stays(i + lane, eqs), in = i + lane < rows, low = j < p.keep;
        const uint32_t h = __ballot_sync(0xffffffffu, in && low && !stay), m = __ballot_sync(0xffffffffu, in && !low && stay);
        const uint32_t ahead = (1u << lane) - 1u;
        if (in && low && !stay) hole_list[holes + __popc(h & ahead)] = j;
        if (in && !low && stay) mover_list[movers + __popc(m & ahead)] = j;
        holes += __popc(h), movers += __popc(m);
    }
    meet();  // the lists are written; movers and holes are equally many
    // Where there are few moves the first warps have their rows, the last their weights, one between the lengths.
    // (A move whose source or target no page backs is not made: the hole keeps its row, weight and position.)
    for (int i = (blocks - me) * THREADS - 1 - tid; i < moves; i += blocks * THREADS) {
        const int s = __ldcg(mover_list + i), d = __ldcg(hole_list + i);
        const float wv = __ldcg(w + s);
        const int pv = __ldcg(pos + s);
        int in_page;
        const int s_e = p.pages.entry(b, s, in_page), d_e = p.pages.entry(b, d, in_page);
        if (p.pages.page(s_e) >= 0 && p.pages.page(d_e) >= 0) w_out[d] = wv, pos_out[d] = pv;
    }
    if (me == blocks - 1 && wid == WARPS / 2) head_done();
    const uint4* const src[2] = {p.pool[0], p.pool[1]};
    const int first = (me * WARPS + wid) * 8, round = blocks * WARPS * 8;
    // lane l < 8: the rows that row l of a round comes from and goes to, read a round ahead
    int s = -1, d = -1;
    auto listed = [&](int m) {
        s = d = -1;
        if (lane < 8 && m + lane < moves) s = __ldcg(mover_list + m + lane), d = __ldcg(hole_list + m + lane);
    };
    listed(first);
#pragma unroll 1
    for (int m0 = first; m0 < moves; m0 += round) {
        uint32_t from = kNoRow, to = kNoRow;
        if (d >= 0) {
            int s_in, d_in;
            const int s_e = p.pages.entry(b, s, s_in), d_e = p.pages.entry(b, d, d_in);  // both loads before a look at either
            const int s_pg = p.pages.page(s_e), d_pg = p.pages.page(d_e);
            if (s_pg >= 0) from = static_cast<uint32_t>((static_cast<long long>(s_pg) * Hkv + h) * p.pages.page_rows + s_in);
            if (d_pg >= 0) to = static_cast<uint32_t>((static_cast<long long>(d_pg) * Hkv + h) * p.pages.page_rows + d_in);
        }
        listed(m0 + round);
        copy_rows8<VPR>(src, p.pool, from, to);
    }
}

}  // namespace e2d2
