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
// and holes, move copies the K and V rows over the whole GPU.
#pragma once

#include <cstdint>

#include "kv_paged.cuh"

namespace e2d2 {

constexpr int kEvictThreads = 1024;

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

// Exclusive prefix of x over the block's threads; *total gets the sum.  Every thread calls it.
__device__ __forceinline__ int block_exclusive_scan(int x, int* wsum, int* total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();  // the previous scan's sums have been read
    if (lane == 31) wsum[wid] = inc;
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < kEvictThreads / 32; ++i) {
        const int s = wsum[i];
        before += i < wid ? s : 0;
        all += s;
    }
    *total = all;
    return before + inc - x;
}

__global__ void __launch_bounds__(kEvictThreads) kv_evict_select_kernel(const __grid_constant__ EvictParams p) {
    __shared__ unsigned int hist[256];
    __shared__ int wsum[kEvictThreads / 32];
    __shared__ unsigned int s_prefix, s_need;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int unit = blockIdx.x, Hkv = p.pages.kv_heads, cap = p.pages.capacity();
    const int b = unit / Hkv, tid = threadIdx.x;
    const int P = ragged_clamp(__ldcg(p.P_dev + b), cap);
    const float* w = p.weight + static_cast<long long>(unit) * cap;
    const int* pos = p.pos + static_cast<long long>(unit) * cap;
    float* w_out = p.weight_out + static_cast<long long>(unit) * cap;
    int* pos_out = p.pos_out + static_cast<long long>(unit) * cap;
    int* ws = p.ws + unit * p.ws_stride;
    const int n_out = P < p.keep ? P : p.keep;
    if (P <= p.keep) {
        if (tid == 0) {
            ws[0] = 0;
            ws[1] = n_out;
        }
        for (int j = tid; j < P; j += kEvictThreads) {
            w_out[j] = w[j];
            pos_out[j] = pos[j];
        }
        return;
    }
    // the first protected position, without overflow for any recent >= 0
    const long long pf = static_cast<long long>(__ldcg(p.tokens + b)) - p.recent;
    const int protect = pf < INT_MIN ? INT_MIN : static_cast<int>(pf);
    // Radix selection of the keep-th largest rank, eight bits a pass: prefix = its leading bits, need = how
    // many rows with that prefix stay.
    unsigned int prefix = 0, need = p.keep;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int j = tid; j < P; j += kEvictThreads) {
            const uint32_t r = evict_rank(w[j], pos[j], protect);
            if (shift == 24 || (r >> (shift + 8)) == prefix) atomicAdd(&hist[(r >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            unsigned int left = need;
            int bin = 255;
            while (bin > 0 && hist[bin] < left) left -= hist[bin--];
            s_prefix = (prefix << 8) | bin;
            s_need = left;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
    }
    // Rows above the threshold stay, and the first `need` rows that equal it.  One row per thread and round,
    // in the order of the rows.
    int eq_seen = 0, holes = 0, movers = 0;
    int* hole_list = ws + 4;
    int* mover_list = hole_list + p.list_rows;
    for (int base = 0; base < P; base += kEvictThreads) {
        const int j = base + tid;
        const uint32_t r = j < P ? evict_rank(w[j], pos[j], protect) : 0u;
        const bool eq = j < P && r == prefix;
        int total;
        const int eq_before = eq_seen + block_exclusive_scan(eq, wsum, &total);
        eq_seen += total;
        const bool kept = j < P && (r > prefix || (eq && eq_before < static_cast<int>(need)));
        const bool hole = j < p.keep && !kept, mover = j >= p.keep && kept;
        const int hi = holes + block_exclusive_scan(hole, wsum, &total);
        holes += total;
        const int mi = movers + block_exclusive_scan(mover, wsum, &total);
        movers += total;
        if (hole) hole_list[hi] = j;
        if (mover) mover_list[mi] = j;
        if (kept && j < p.keep) {
            w_out[j] = w[j];
            pos_out[j] = pos[j];
        }
    }
    __syncthreads();  // the lists are written; movers and holes are equally many
    for (int i = tid; i < movers; i += kEvictThreads) {
        w_out[hole_list[i]] = w[mover_list[i]];
        pos_out[hole_list[i]] = pos[mover_list[i]];
    }
    if (tid == 0) {
        ws[0] = movers;
        ws[1] = n_out;
    }
}

// blockIdx.y: (entry, kv head).  A row of K or V is vec_per_row threads of 16 bytes each.
__global__ void __launch_bounds__(256) kv_evict_move_kernel(const __grid_constant__ EvictParams p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int unit = blockIdx.y, Hkv = p.pages.kv_heads;
    const int b = unit / Hkv, h = unit % Hkv;
    const int* ws = p.ws + unit * p.ws_stride;
    const int* hole_list = ws + 4;
    const int* mover_list = hole_list + p.list_rows;
    const long long total = static_cast<long long>(ws[0]) * 2 * p.vec_per_row;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        const int move = static_cast<int>(i / (2 * p.vec_per_row));
        const int rest = static_cast<int>(i - static_cast<long long>(move) * 2 * p.vec_per_row);
        const int which = rest >= p.vec_per_row, vec = rest - which * p.vec_per_row;
        const long long s = p.pages.pool_row(b, h, mover_list[move]), d = p.pages.pool_row(b, h, hole_list[move]);
        if (s >= 0 && d >= 0) p.pool[which][d * p.vec_per_row + vec] = p.pool[which][s * p.vec_per_row + vec];
    }
    // the lengths come last: P_out may be P_dev, which the first launch read
    if (h == 0 && blockIdx.x == 0 && threadIdx.x == 0) p.P_out[b] = ws[1];
}

}  // namespace e2d2
