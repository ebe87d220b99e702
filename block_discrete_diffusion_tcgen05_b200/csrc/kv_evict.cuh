// kv_evict.cuh -- eviction from a KV cache by accumulated attention weight.
//
// Per (entry, kv head): of the P rows, `keep` stay.  Rows at positions >= tokens - recent come first, then
// the rows by decreasing weight, ties to the lowest row.  Kept rows below `keep` stay where they are; the
// i-th kept row at or past `keep` (a mover) goes to the i-th row below `keep` that is not kept (a hole), so
// a call moves no more rows than it must, and sources (at or past keep) and targets (below it) never
// overlap.  Attention over the prefix does not depend on the order of its rows; pos says which token each
// one is.
//
// Two launches: select (one block per (entry, kv head)) finds the kept rows and writes the lists of movers
// and holes, move copies the K and V rows over the whole GPU.  Select reads 8 bytes a row once, keeps the rows'
// ranks in shared memory (up to 32768 rows), finds the keep-th largest by its four bytes in turn (a histogram of 256
// bins each) and turns "stays" into one bit a row, from whose counts every row's place in its list follows: no
// sort, and no atomics but the histograms' counts.
#pragma once

#include <cstdint>

#include "kv_paged.cuh"

namespace e2d2 {

constexpr int kEvictRows = 32768;  // rows whose ranks (and bits) are held in shared memory at a time

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
    int* ws;              // per unit: count, kept length, 2 unused, then list_rows holes, list_rows movers
    int batch, keep, recent, vec_per_row;
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

// Exclusive prefix of (x, y) over the block's threads, their totals in *tx, *ty.  Every thread calls it.
template <int THREADS>
__device__ __forceinline__ int2 block_exclusive_scan(int x, int y, int2* wsum, int2* total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int ix = x, iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, ix, o), b = __shfl_up_sync(0xffffffffu, iy, o);
        if (lane >= o) ix += a, iy += b;
    }
    __syncthreads();  // the previous scan's sums have been read
    if (lane == 31) wsum[wid] = make_int2(ix, iy);
    __syncthreads();
    int2 before = make_int2(ix - x, iy - y), all = make_int2(0, 0);
#pragma unroll 8
    for (int i = 0; i < THREADS / 32; ++i) {
        const int2 s = wsum[i];
        if (i < wid) before.x += s.x, before.y += s.y;
        all.x += s.x, all.y += s.y;
    }
    *total = all;
    return before;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) kv_evict_select_kernel(const __grid_constant__ EvictParams p) {
    constexpr int WARPS = THREADS / 32;
    __shared__ unsigned int hist[256];
    __shared__ int2 wsum[WARPS];
    __shared__ unsigned int s_pick[3];                // leading bytes, rows of them that stay, rows that have them
    __shared__ uint32_t kept_bits[kEvictRows / 32];
    __shared__ int2 word_at[kEvictRows / 32];         // holes and movers before each 32 rows
    extern __shared__ uint32_t ranks[];               // [rank_rows]
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int unit = blockIdx.x, Hkv = p.pages.kv_heads, cap = p.pages.capacity();
    const int b = unit / Hkv, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int P = ragged_clamp(__ldcg(p.P_dev + b), cap);
    const long long row0 = static_cast<long long>(unit) * cap;
    const float* w = p.weight + row0;
    const int* pos = p.pos + row0;
    float* w_out = p.weight_out + row0;
    int* pos_out = p.pos_out + row0;
    int* ws = p.ws + unit * p.ws_stride;
    if (P <= p.keep) {
        if (tid == 0) {
            ws[0] = 0;
            ws[1] = P;
        }
        if (w_out != w || pos_out != pos)
            for (int j = tid; j < P; j += THREADS) {
                w_out[j] = w[j];
                pos_out[j] = pos[j];
            }
        return;
    }
    // the first protected position, without overflow for any recent >= 0
    const long long pf = static_cast<long long>(__ldcg(p.tokens + b)) - p.recent;
    const int protect = pf < INT_MIN ? INT_MIN : static_cast<int>(pf);
    const bool held = P <= p.rank_rows;
    auto rank_of = [&](int j) { return held ? ranks[j] : evict_rank(__ldcg(w + j), __ldcg(pos + j), protect); };
    if (tid < 256) hist[tid] = 0;
    for (int i = tid + THREADS; i < 256; i += THREADS) hist[i] = 0;
    __syncthreads();

    // The keep-th largest rank, a byte a pass: prefix = its leading bytes, need = how many rows with that prefix
    // stay.  The first pass also fills the ranks.
    unsigned int prefix = 0, need = p.keep, equal = 0;
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
#pragma unroll 4
        for (int j = tid; j < P; j += THREADS) {
            uint32_t r;
            if (shift == 24) {
                r = evict_rank(__ldcg(w + j), __ldcg(pos + j), protect);
                if (held) ranks[j] = r;
            } else {
                r = rank_of(j);
            }
            if (shift == 24 || (r >> (shift + 8)) == prefix) atomicAdd(&hist[(r >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (wid == 0) {
            // lane l: bins 255 - 8 l down to 248 - 8 l; the bin where the count from above reaches need
            unsigned int mine[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += mine[i] = hist[255 - 8 * lane - i];
            unsigned int inc = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            unsigned int above = inc - sum;
            // need = 0 (keep = 0): no bin qualifies, the largest one is taken and nothing of it stays
            const unsigned int reach = __ballot_sync(0xffffffffu, inc >= need);
            if (lane == __ffs(reach) - 1) {
                int i = 0;
                while (i < 7 && above + mine[i] < need) above += mine[i++];
                s_pick[0] = (prefix << 8) | static_cast<unsigned int>(255 - 8 * lane - i);
                s_pick[1] = need - above;
                s_pick[2] = mine[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) hist[255 - 8 * lane - i] = 0;
        }
        __syncthreads();
        prefix = s_pick[0];
        need = s_pick[1];
        equal = s_pick[2];
    }
    // Rows above the threshold stay, and the first `need` of the rows that equal it.
    int* hole_list = ws + 4;
    int* mover_list = hole_list + p.list_rows;
    int eq_seen = 0;
    int2 seen = make_int2(0, 0);  // holes, movers
    const bool copy = w_out != w || pos_out != pos;
#pragma unroll 1
    for (int base = 0; base < P; base += kEvictRows) {
        const int rows = min(P - base, kEvictRows), words = (rows + 31) / 32;
        const int per = (words + WARPS - 1) / WARPS, w0 = min(wid * per, words), w1 = min(w0 + per, words);
        int eq_before = 0;
        if (equal != need) {  // ties at the threshold: which of them are the first
            int mine = 0;
            for (int k = w0; k < w1; ++k) {
                const int j = base + 32 * k + lane;
                mine += __popc(__ballot_sync(0xffffffffu, j < P && rank_of(j) == prefix));
            }
            int2 all;
            eq_before = eq_seen + block_exclusive_scan<THREADS>(lane == 0 ? mine : 0, 0, wsum, &all).x;
            eq_before = __shfl_sync(0xffffffffu, eq_before, 0);
            eq_seen += all.x;
        }
        __syncthreads();  // the last round's bits have been read
#pragma unroll 2
        for (int k = w0; k < w1; ++k) {
            const int j = base + 32 * k + lane;
            const uint32_t r = j < P ? rank_of(j) : 0u;
            const bool eq = j < P && r == prefix;
            const uint32_t eqs = __ballot_sync(0xffffffffu, eq);
            const bool stay = (j < P && r > prefix) ||
                              (eq && (equal == need || eq_before + __popc(eqs & ((1u << lane) - 1u)) < static_cast<int>(need)));
            eq_before += __popc(eqs);
            const uint32_t bits = __ballot_sync(0xffffffffu, stay);
            if (lane == 0) kept_bits[k] = bits;
        }
        __syncthreads();
        for (int k0 = 0; k0 < words; k0 += THREADS) {
            const int k = k0 + tid, j = base + 32 * k;
            int2 n = make_int2(0, 0), all;
            if (k < words) {
                // rows of the word below keep, a mask
                const uint32_t low = j + 32 <= p.keep ? 0xffffffffu : (j >= p.keep ? 0u : (1u << (p.keep - j)) - 1u);
                n = make_int2(__popc(~kept_bits[k] & low), __popc(kept_bits[k] & ~low));
            }
            const int2 at = block_exclusive_scan<THREADS>(n.x, n.y, wsum, &all);
            if (k < words) word_at[k] = make_int2(seen.x + at.x, seen.y + at.y);
            seen.x += all.x, seen.y += all.y;
        }
        __syncthreads();
#pragma unroll 2
        for (int k = w0; k < w1; ++k) {
            const int j = base + 32 * k + lane;
            const uint32_t bits = kept_bits[k], below = (1u << lane) - 1u;
            const uint32_t low = j - lane + 32 <= p.keep ? 0xffffffffu : (j - lane >= p.keep ? 0u : (1u << (p.keep - (j - lane))) - 1u);
            const int2 at = word_at[k];
            const bool stay = (bits >> lane) & 1u;
            if (j < p.keep && !stay) hole_list[at.x + __popc(~bits & low & below)] = j;
            if (j >= p.keep && stay) mover_list[at.y + __popc(bits & ~low & below)] = j;
            if (copy && j < p.keep && stay) {
                w_out[j] = __ldcg(w + j);
                pos_out[j] = __ldcg(pos + j);
            }
        }
    }
    __syncthreads();  // the lists are written; movers and holes are equally many
    for (int i = tid; i < seen.y; i += THREADS) {
        const int s = mover_list[i], d = hole_list[i];
        w_out[d] = w[s];
        pos_out[d] = pos[s];
    }
    if (tid == 0) {
        ws[0] = seen.y;
        ws[1] = p.keep;
    }
}

// blockIdx.y: (entry, kv head).  A warp takes eight moves at a time: lane l looks up where row l comes from and goes
// to, then all of its rows are loaded before the first is stored.  VPR: 16-byte vectors per row; K and V of one row
// (two, four at smaller head dims) are a warp's 32 vectors.
template <int VPR>
__global__ void __launch_bounds__(256) kv_evict_move_kernel(const __grid_constant__ EvictParams p) {
    constexpr int RPS = 16 / VPR, STEPS = 8 / RPS;  // rows per step, steps per eight moves
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int unit = blockIdx.y, Hkv = p.pages.kv_heads, lane = threadIdx.x & 31;
    const int b = unit / Hkv, h = unit % Hkv;
    const int* ws = p.ws + unit * p.ws_stride;
    const int* hole_list = ws + 4;
    const int* mover_list = hole_list + p.list_rows;
    const int moves = __ldcg(ws);
    const int which = (lane / VPR) & 1, vec = lane % VPR, sub = lane / (2 * VPR);
    uint4* pool = p.pool[which];
    for (int m0 = (blockIdx.x * 8 + threadIdx.x / 32) * 8; m0 < moves; m0 += gridDim.x * 64) {
        long long from = -1, to = -1;
        if (lane < 8 && m0 + lane < moves) {
            from = p.pages.pool_row(b, h, __ldcg(mover_list + m0 + lane));
            to = p.pages.pool_row(b, h, __ldcg(hole_list + m0 + lane));
        }
        uint4 x[STEPS];
        long long d[STEPS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const long long s = __shfl_sync(0xffffffffu, from, k * RPS + sub);
            d[k] = __shfl_sync(0xffffffffu, to, k * RPS + sub);
            if (s < 0) d[k] = -1;
            if (d[k] >= 0) x[k] = __ldcg(pool + s * VPR + vec);
        }
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
            if (d[k] >= 0) pool[d[k] * VPR + vec] = x[k];
    }
    // the lengths come last: P_out may be P_dev, which the first launch read
    if (h == 0 && blockIdx.x == 0 && threadIdx.x == 0) p.P_out[b] = __ldcg(ws + 1);
}

}  // namespace e2d2
