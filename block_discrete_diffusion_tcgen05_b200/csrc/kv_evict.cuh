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
// ranks in shared memory (up to 32768 rows), finds the keep-th largest by 11, 11 and 10 bits in turn (histograms
// in shared memory; eleven bits tell weights apart that share an exponent, so few lanes meet in a bin) and turns "stays" into one bit a row, from whose counts every row's place in its list follows: no
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
    __shared__ unsigned int hist[2048];
    __shared__ int2 wsum[WARPS];
    __shared__ unsigned int s_pick[3];                // leading bits, rows of them that stay, rows that have them
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
    for (int i = tid; i < 2048; i += THREADS) hist[i] = 0;
    __syncthreads();

    // The keep-th largest rank, 11, 11 and 10 bits a pass: prefix = its leading bits, need = how many rows with that
    // prefix stay.  The first pass also fills the ranks.
    unsigned int prefix = 0, need = p.keep, equal = 0;
    auto count = [&](bool in, uint32_t bin) {
        // equal weights (a fresh cache's zeros) would queue at one bin: a warp of one bin counts once
        const unsigned int lanes = __ballot_sync(0xffffffffu, in);
        if (lanes == 0) return;
        const int lead = __ffs(lanes) - 1;
        const uint32_t first = __shfl_sync(0xffffffffu, bin, lead);
        if (__all_sync(0xffffffffu, !in || bin == first)) {
            if (lane == lead) atomicAdd(&hist[bin], __popc(lanes));
        } else if (in) {
            atomicAdd(&hist[bin], 1u);
        }
    };
    constexpr int BATCH = 8;
#pragma unroll 1
    for (int j0 = 0; j0 < P; j0 += BATCH * THREADS) {
        float wv[BATCH];
        int pv[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int j = j0 + k * THREADS + tid;
            wv[k] = j < P ? __ldcg(w + j) : 0.f;
            pv[k] = j < P ? __ldcg(pos + j) : 0;
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int j = j0 + k * THREADS + tid;
            const uint32_t r = evict_rank(wv[k], pv[k], protect);
            if (held && j < P) ranks[j] = r;
            count(j < P, r >> 21);
        }
    }
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
        if (pass > 0) {
#pragma unroll 4
            for (int j = tid; j < (P + 31) / 32 * 32; j += THREADS) {
                const uint32_t r = j < P ? rank_of(j) : 0u;
                count(j < P && (r >> (shift + bits)) == prefix, (r >> shift) & ((1u << bits) - 1u));
            }
        }
        __syncthreads();
        // bins from the largest down, BINS of them per thread: the one where the count from above reaches need
        constexpr int BINS = 2048 / THREADS;
        unsigned int mine[BINS], sum = 0;
#pragma unroll
        for (int i = 0; i < BINS; ++i) {
            sum += mine[i] = hist[2047 - BINS * tid - i];
            hist[2047 - BINS * tid - i] = 0;
        }
        int2 all;
        unsigned int above = block_exclusive_scan<THREADS>(static_cast<int>(sum), 0, wsum, &all).x;
        // need = 0 (keep = 0): the first thread takes its first bin, and nothing of it stays
        if (need == 0 ? tid == 0 : (above < need && need <= above + sum)) {
            int i = 0;
            while (i < BINS - 1 && above + mine[i] < need) above += mine[i++];
            s_pick[0] = (prefix << bits) | ((2047u - BINS * tid - i) & ((1u << bits) - 1u));
            s_pick[1] = need == 0 ? 0 : need - above;
            s_pick[2] = mine[i];
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
// to.  VPR: 16-byte vectors per row.
template <int VPR>
__global__ void __launch_bounds__(256) kv_evict_move_kernel(const __grid_constant__ EvictParams p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int unit = blockIdx.y, Hkv = p.pages.kv_heads, lane = threadIdx.x & 31;
    const int b = unit / Hkv, h = unit % Hkv;
    const int* ws = p.ws + unit * p.ws_stride;
    const int* hole_list = ws + 4;
    const int* mover_list = hole_list + p.list_rows;
    const int moves = __ldcg(ws);
    const uint4* const src[2] = {p.pool[0], p.pool[1]};
    for (int m0 = (blockIdx.x * 8 + threadIdx.x / 32) * 8; m0 < moves; m0 += gridDim.x * 64) {
        long long from = -1, to = -1;
        if (lane < 8 && m0 + lane < moves) {
            from = p.pages.pool_row(b, h, __ldcg(mover_list + m0 + lane));
            to = p.pages.pool_row(b, h, __ldcg(hole_list + m0 + lane));
        }
        copy_rows8<VPR>(src, p.pool, from, to);
    }
    // the lengths come last: P_out may be P_dev, which the first launch read
    if (h == 0 && blockIdx.x == 0 && threadIdx.x == 0) p.P_out[b] = __ldcg(ws + 1);
}

}  // namespace e2d2
