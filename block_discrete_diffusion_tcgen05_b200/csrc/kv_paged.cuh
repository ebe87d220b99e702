// kv_paged.cuh -- what every call on a paged KV cache shares (the view of the pool through the page
// table), and the append to it.
//
// A pool holds num_pages pages of page_rows rows for every kv head, [num_pages][kv_heads][page_rows][d];
// entry b's row r is row r mod page_rows of page table[b][r / page_rows].  Without a table the pool is
// one contiguous cache per entry: entry b is page b, and a page holds the entry's whole capacity.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "fmha_sm100.cuh"
#include "ptx_sm100.cuh"

namespace e2d2 {

// Bit of the device error word: a page id outside the pool was met below an entry's length.
constexpr unsigned int kErrBadPage = 4u;
constexpr int kPagedMaxBatch = 1024;  // entries of a call (the prefix table of its schedule)

// What a call reads (lengths, tables, queries, weights) may come from the kernel ahead of it on the stream,
// which it overlaps until griddepcontrol.wait: such values are read through L2 (ld.cg), never as read-only.
struct PageView {
    const int* table;  // [batch][max_pages], null: entry b is page b
    int num_pages, page_rows, max_pages;
    int kv_heads;
    // r / page_rows for r < 2^30 as a product: with 2^l the power of two from page_rows on, div_mul = ceil(2^(30+l) / page_rows),
    // whose excess over the quotient, less than 2^l / page_rows, moves r div_mul / 2^(30+l) by less than 1 / page_rows.
    // (The division is some twenty instructions; every key of the softmax looks its page up.)
    unsigned div_mul, div_shift;  // div_shift = l - 2
    unsigned int* err;

    __device__ __forceinline__ int capacity() const { return max_pages * page_rows; }

    // The table's entry for row r of entry b (r inside the capacity), and the row inside the page.  Loaded, not
    // looked at: what page() makes of it can wait until the load is back.
    __device__ __forceinline__ int entry(int b, int r, int& in_page) const {
        in_page = r;
        if (table == nullptr) return b;
        const int at = __umulhi(static_cast<unsigned>(r), div_mul) >> div_shift;
        in_page = r - at * page_rows;
        return __ldcg(table + static_cast<size_t>(b) * max_pages + at);
    }
    // The page that an entry names; -1, with the error recorded, if it is none of the pool.  Nothing is read or
    // written through such an entry.
    __device__ __forceinline__ int page(int e) const {
        if (static_cast<unsigned>(e) < static_cast<unsigned>(num_pages)) return e;
        atomicOr(err, kErrBadPage);
        return -1;
    }

    // Row of the pool (in rows of d elements) that holds row r of entry b, head h; -1 as above.  64 bits:
    // a pool has more elements than 32 bits count.
    __device__ __forceinline__ long long pool_row(int b, int h, int r) const {
        int in_page;
        const int pg = page(entry(b, r, in_page));
        return pg < 0 ? -1 : (static_cast<long long>(pg) * kv_heads + h) * page_rows + in_page;
    }
};

// wait_bar_warp for a pipeline's steady state, where most waits are short and one follows the other: a few sleeping
// attempts (the thread wakes when the phase completes, or after 50 us) before the bounded wait, whose limit and
// clock cost a trip to global memory -- paid at every stage, that trip alone held a loader to one stage a
// microsecond.
__device__ __forceinline__ bool wait_stage_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned int* err) {
    bool ok = ptx::mbar_try_wait(bar, parity);
    for (int i = 0; i < 4 && !ok; ++i) ok = ptx::mbar_try_wait_sleep(bar, parity, 50000u);
    if (__all_sync(0xffffffffu, ok)) return true;
    return wait_bar_warp(bar, parity, abort_flag, err);
}

// The work of a call as one stream of places: entry b takes units * places(P[b]) of them, the entries one after the
// other (below 2^31 in all, the host sees to it).  Every warp works it out for itself, a lane per entry, 32 entries
// at a time: no shared memory, no barrier.
template <class Places>
struct EntryStream {
    const int* P_dev;
    int batch, cap, lane;
    unsigned units, lead;  // lead: places of every unit on top of places(P)
    Places places;
    int P;                // of lane's entry in the batch of 32 at hand
    unsigned n;
    unsigned total;       // places in all
    bool equal;           // every entry takes as many

    __device__ EntryStream(const int* lengths, int b, int capacity, unsigned units_per_entry, Places f)
        : P_dev(lengths), batch(b), cap(capacity), lane(threadIdx.x & 31), units(units_per_entry), lead(0), places(f) {
        unsigned sum = 0, most = 0;
        for (int base = 0; base < batch; base += 32) {
            load(base);
            sum += __reduce_add_sync(0xffffffffu, n);
            most = max(most, __reduce_max_sync(0xffffffffu, n));
        }
        total = sum * units;
        equal = sum == most * batch;
    }
    __device__ void load(int base) {
        P = base + lane < batch ? ragged_clamp(__ldcg(P_dev + base + lane), cap) : 0;
        n = base + lane < batch ? places(P) : 0;
    }
    // The entry that holds place pos < total, the places before it and its length.
    __device__ void find(unsigned pos, int& entry, unsigned& before, int& length) {
        before = 0;
        for (int base = 0;; base += 32) {
            if (batch > 32) load(base);
            const unsigned mine = base + lane < batch ? n + lead : 0;
            unsigned inc = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + inc * units > pos);
            if (past != 0 || base + 32 >= batch) {
                const int at = past != 0 ? __ffs(past) - 1 : 31;
                entry = base + at;
                before += __shfl_sync(0xffffffffu, inc - mine, at) * units;
                length = __shfl_sync(0xffffffffu, P, at);
                return;
            }
            before += __shfl_sync(0xffffffffu, inc, 31) * units;
        }
    }
};

template <class Places>
__device__ __forceinline__ EntryStream<Places> entry_stream(const int* P_dev, int batch, int cap, unsigned units, Places f) {
    return EntryStream<Places>(P_dev, batch, cap, units, f);
}

// The test hook's delay, read while the previous kernel still runs; the producer sleeps before its first load.
__device__ __forceinline__ bool producer_delay_set() {
    return *reinterpret_cast<volatile unsigned long long*>(&g_test_producer_delay_ns) != 0;
}

// One arrival for a warp whose lanes are all done (32 arrivals at one barrier queue there).
__device__ __forceinline__ void mbar_arrive_warp(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
}

// Copies rows of K and V, eight at a time, by one warp: lane l < 8 gives the rows (of VPR 16-byte vectors) that move
// l reads and writes, kNoRow for none (a row number fits in 32 bits: 2^32 rows of d = 32 are more than the memory).  K
// and V of one row (of two, four at smaller head dims) are the warp's 32 vectors; all of the eight are loaded before
// the first is stored.
constexpr uint32_t kNoRow = 0xffffffffu;
template <int VPR>
__device__ __forceinline__ void copy_rows8(const uint4* const (&src)[2], uint4* const (&dst)[2], uint32_t from, uint32_t to) {
    constexpr int RPS = 16 / VPR, STEPS = 8 / RPS;  // rows per step, steps
    const int lane = threadIdx.x & 31, which = (lane / VPR) & 1, vec = lane % VPR, sub = lane / (2 * VPR);
    const uint4* s_base = (which ? src[1] : src[0]) + vec;
    uint4* d_base = (which ? dst[1] : dst[0]) + vec;
    if (from == kNoRow) to = kNoRow;
    uint4 x[STEPS];
    uint32_t d[STEPS];
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
        const uint32_t s = __shfl_sync(0xffffffffu, from, k * RPS + sub);
        d[k] = __shfl_sync(0xffffffffu, to, k * RPS + sub);
        if (d[k] != kNoRow) x[k] = __ldcg(s_base + static_cast<size_t>(s) * VPR);
    }
#pragma unroll
    for (int k = 0; k < STEPS; ++k)
        if (d[k] != kNoRow) d_base[static_cast<size_t>(d[k]) * VPR] = x[k];
}

struct PagedAppendParams {
    PageView pages;
    uint4* pool[2];       // K, V pools
    const uint4* src[2];  // new rows [B][Hkv][S_new][D]
    const int* P_dev;
    float* weight;        // [B][Hkv][capacity] or null: the new rows' accumulated weight becomes 0,
    int* pos;             // [B][Hkv][capacity] or null: their position tokens[b] + i
    const int* tokens;
    int batch, S_new;
};

// A pure copy, HBM-bound: a warp per eight new rows, grid-stride.  4 prompts of 4095 tokens (135 MB read and written)
// take 26.3 us, 5.1 TB/s; one 16-byte vector per thread and step, with its row looked up by every thread, took 44 us.
// Four blocks per SM: five spill (32 us).
template <int VPR>
__global__ void __launch_bounds__(256, 4) kv_append_paged_kernel(const __grid_constant__ PagedAppendParams a) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();  // the previous kernel may still read the pool or write the new rows
    const int Hkv = a.pages.kv_heads, cap = a.pages.capacity(), lane = threadIdx.x & 31;
    const long long total = static_cast<long long>(a.batch) * Hkv * a.S_new;
    for (long long r0 = (blockIdx.x * 8ll + threadIdx.x / 32) * 8; r0 < total; r0 += gridDim.x * 64ll) {
        const long long from = r0 + lane;
        uint32_t to = kNoRow;
        if (lane < 8 && from < total) {
            const int unit = static_cast<int>(from / a.S_new), s = static_cast<int>(from - static_cast<long long>(unit) * a.S_new);
            const int b = unit / Hkv, h = unit - b * Hkv;
            const long long r = static_cast<long long>(ragged_clamp(__ldcg(a.P_dev + b), cap)) + s;
            // rows past the capacity, and those that no page backs, are not written; nor are their weights and positions
            if (r < cap) to = static_cast<uint32_t>(a.pages.pool_row(b, h, static_cast<int>(r)));  // -1: kNoRow
            if (to != kNoRow && a.weight != nullptr) {
                const long long w = static_cast<long long>(unit) * cap + r;
                a.weight[w] = 0.f;
                a.pos[w] = __ldcg(a.tokens + b) + s;
            }
        }
        copy_rows8<VPR>(a.src, a.pool, static_cast<uint32_t>(from), to);
    }
}

}  // namespace e2d2
