// kv_weigh.cuh -- accumulated attention weight of a cache's rows: with the lse of an attention call,
//
//   weight_out_j = weight_j + sum_i exp(scale q_i . k_j - lse_i)      (i over the G S rows that read kv head h)
//
// K is read once and nothing else is large, so the kernel is bound by HBM for up to some 160 query rows (then by
// the exponentials: 16 a clock and SM against 22 bytes of K).  The scores are taken transposed, S^T = K Q^T with
// 128 keys on the tensor-memory lanes: a thread of the epilogue holds one key's scores, so the sum over the
// query rows is a sum in its own registers -- no shuffles, no atomics, one order -- and the normaliser is known
// (lse), so there is no maximum to track.
//
// Warp 0 loads (a ring of key tiles of 128 rows, in boxes that end where pages do; Q once per unit), warp 1
// issues the products into two buffers of tensor memory, and two warpgroups take the tiles in turn: one reads
// its scores while the other's are computed.  The tiles of all (entry, kv head) units form one stream cut
// evenly over a persistent grid.  Up to 32 query rows two blocks share an SM, so one starts or changes units while the
// other streams: 32 blocks of 16 tokens over 2064 rows (32 query rows per head) take 28 us, 5.0 TB/s, against 32 us
// with one block per SM.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "kv_paged.cuh"

namespace e2d2 {

constexpr int kWeighThreads = 384;  // 12 warps: loads, products, two idle, two epilogue warpgroups
constexpr int kWeighKeys = 128;
constexpr int kWeighMaxRows = 256;  // query rows of one launch (columns of one product)

struct alignas(64) WeighParams {
    CUtensorMap tm_k;     // pool: 3D {D, page_rows, num_pages * Hkv}, boxes of box_rows
    CUtensorMap tm_q;     // 2D {D, B * Hq * S}, boxes of 16 rows
    PageView pages;
    const int* P_dev;
    const float* lse;     // [B][Hq][S]
    const float* weight;  // [B][Hkv][capacity]
    float* weight_out;
    unsigned int* err;
    int batch, box_rows;
    int rows, row0, n;    // query rows per kv head (G * S); this launch takes rows row0.., n of them
    float scale_log2;
};

// N: columns that shared and tensor memory are laid out for (the launch's rows rounded up).
template <int D_, int N_>
struct WeighCfg {
    static constexpr int D = D_, N = N_;
    static constexpr int RB = D * 2 < 128 ? D * 2 : 128;  // bytes per row of one column chunk
    static constexpr int NCH = D * 2 / RB;
    static constexpr uint32_t SWZ = RB == 128 ? 2u : 4u;
    static constexpr int QCHUNK = N * RB, Q_BYTES = NCH * QCHUNK;
    static constexpr int KCHUNK = kWeighKeys * RB, K_BYTES = NCH * KCHUNK;
    static constexpr int CTAS = N == 32 ? 2 : 1;  // blocks per SM
    static constexpr int QB = N == 64 ? 2 : 1;
    static constexpr int FIT = ((CTAS == 2 ? 109 : 216) * 1024 - QB * Q_BYTES) / K_BYTES;
    static constexpr int NST = FIT < 8 ? FIT : 8;
    static constexpr uint32_t TMEM_COLS = 2 * N < 32 ? 32u : 2u * N;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + QB * Q_BYTES;
    static constexpr int OFF_BAR = OFF_K + NST * K_BYTES;
    // k_full[NST], k_empty[NST], q_full[QB], q_empty[QB], s_full[2], s_free[2], drain, done
    static constexpr int NBAR = 2 * NST + 2 * QB + 6;
    static constexpr int OFF_LSE = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;  // float [8 warps][N]
    static constexpr int OFF_MISC = OFF_LSE + 8 * N * 4;                       // holder, abort, plan
    static constexpr int BYTES = OFF_MISC + 8 + 24;
    static constexpr int ALLOC = (BYTES + 1023) / 1024 * 1024 + 1024;
    static_assert(NST >= 2 && ALLOC <= 232448 && TMEM_COLS <= 512, "shared and tensor memory");
};

__device__ __forceinline__ unsigned weigh_tiles(int P) { return (P + kWeighKeys - 1) / kWeighKeys; }

// A block's place in the stream of tiles, worked out by one warp for all.
struct WeighPlan {
    unsigned left;
    int b, h, P, t;
};

__device__ __forceinline__ void weigh_plan(const WeighParams& p, WeighPlan* out) {
    auto stream = entry_stream(p.P_dev, p.batch, p.pages.capacity(), p.pages.kv_heads, [](int rows) { return weigh_tiles(rows); });
    WeighPlan n;
    const unsigned q = stream.total / gridDim.x, r = stream.total % gridDim.x, c = blockIdx.x;
    const unsigned first = c * q + c * r / gridDim.x;
    n.left = (c + 1) * q + (c + 1) * r / gridDim.x - first;
    n.b = n.h = n.P = n.t = 0;
    if (n.left > 0) {
        unsigned before;
        stream.find(first, n.b, before, n.P);
        const unsigned tiles = weigh_tiles(n.P);
        n.h = (first - before) / tiles;
        n.t = static_cast<int>(first - before - n.h * tiles) - 1;
    }
    if ((threadIdx.x & 31) == 0) *out = n;
}

// Walks the tiles of this block: unit (entry b, kv head h), key tile t of it.
struct WeighWalk {
    const WeighParams& p;
    unsigned left;   // tiles still to come
    int b, h, P, tiles;
    int unit, t;     // the current tile's unit (b * Hkv + h) and index

    __device__ WeighWalk(const WeighParams& prm, const WeighPlan& n)
        : p(prm), left(n.left), b(n.b), h(n.h), P(n.P), tiles(weigh_tiles(n.P)), unit(0), t(n.t) {}
    // Moves to the next tile; false at the end.
    __device__ bool next() {
        if (left == 0) return false;
        --left;
        if (++t == tiles) {
            t = 0;
            if (++h == p.pages.kv_heads) {
                h = 0;
                do {
                    ++b;
                    P = ragged_clamp(__ldcg(p.P_dev + b), p.pages.capacity());
                    tiles = weigh_tiles(P);
                } while (tiles == 0);  // a tile is left, so an entry with rows follows
            }
        }
        unit = b * p.pages.kv_heads + h;
        return true;
    }
};

template <int D, int N>
__global__ void __launch_bounds__(kWeighThreads, WeighCfg<D, N>::CTAS) kv_weigh_kernel(const __grid_constant__ WeighParams p) {
    using C = WeighCfg<D, N>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* k_empty = k_full + C::NST;
    uint64_t* q_full = k_empty + C::NST;
    uint64_t* q_empty = q_full + C::QB;
    uint64_t* s_full = q_empty + C::QB;
    uint64_t* s_free = s_full + 2;
    uint64_t* drain = s_free + 2;
    uint64_t* done = drain + 1;
    uint32_t* holder = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

    ptx::griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NST; ++i) ptx::mbar_init(&k_full[i], 1), ptx::mbar_init(&k_empty[i], 1);
        for (int i = 0; i < C::QB; ++i) ptx::mbar_init(&q_full[i], 1), ptx::mbar_init(&q_empty[i], 1);
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&s_full[i], 1), ptx::mbar_init(&s_free[i], 4);
        ptx::mbar_init(drain, 1);
        ptx::mbar_init(done, 8);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(holder, C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    const bool delayed = warp == 0 && producer_delay_set();
    ptx::griddep_wait();  // inputs are read after the previous kernel on the stream has finished
    const int cap = p.pages.capacity(), Hkv = p.pages.kv_heads;
    WeighPlan* plan = reinterpret_cast<WeighPlan*>(smem + C::OFF_MISC + 8);
    if (warp == 0) weigh_plan(p, plan);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *holder;
    const int n16 = round16(p.n);

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        // Lane j looks up and loads box j of a tile; the next tile's look-up is done while this one waits.
        if (lane == 0) {
            ptx::tma_prefetch_desc(&p.tm_k);
            ptx::tma_prefetch_desc(&p.tm_q);
        }
        if (delayed) test_producer_delay();
        const int boxes = kWeighKeys / p.box_rows;
        WeighWalk walk(p, *plan);
        // A tile ahead of the one being loaded: its unit, and lane's box of it (row in the page, -1 for none; the
        // table's entry, on its way).
        struct Ahead {
            bool more;
            int unit, y, e;
        };
        auto look_up = [&]() {
            Ahead a;
            a.more = walk.next();
            a.unit = walk.unit;
            a.y = -1;
            a.e = 0;
            const int r = walk.t * kWeighKeys + lane * p.box_rows;
            if (a.more && lane < boxes && r < walk.P) a.e = p.pages.entry(walk.b, r, a.y);
            return a;
        };
        uint32_t it = 0, units = 0;
        int have = -1;
        bool ok = true;
        Ahead one = look_up(), two = look_up();
        while (one.more) {
            const Ahead now = one;
            one = two;
            two = look_up();
            if (now.unit != have) {
                const uint32_t qb = units % C::QB;
                ok = wait_stage_warp(&q_empty[qb], ((units / C::QB) & 1) ^ 1, abort_flag, p.err);
                if (!ok) break;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(&q_full[qb], n16 * D * 2);
                    const int row = now.unit * p.rows + p.row0;  // packed rows of a unit are contiguous
                    for (int ch = 0; ch < C::NCH; ++ch)
                        for (int r = 0; r < n16; r += 16)
                            ptx::tma_load_2d(&p.tm_q, &q_full[qb], smem + C::OFF_Q + qb * C::Q_BYTES + ch * C::QCHUNK + r * C::RB,
                                             ch * 64, row + r);
                }
                __syncwarp();
                ++units;
                have = now.unit;
            }
            const int cy = now.y;
            int cz = now.unit;
            if (cy >= 0 && p.pages.table != nullptr) {
                const int pg = p.pages.page(now.e);
                cz = (pg < 0 ? p.pages.num_pages : pg) * Hkv + (pg < 0 ? 0 : now.unit % Hkv);  // past the pool: zeros
            }
            const uint32_t st = it % C::NST;
            ok = wait_stage_warp(&k_empty[st], ((it / C::NST) & 1) ^ 1, abort_flag, p.err);
            if (!ok) break;
            const int n = __popc(__ballot_sync(0xffffffffu, cy >= 0));
            if (lane == 0) ptx::mbar_arrive_expect_tx(&k_full[st], static_cast<uint32_t>(n) * p.box_rows * D * 2);
            __syncwarp();
            if (cy >= 0)
                for (int ch = 0; ch < C::NCH; ++ch)
                    ptx::tma_load_3d(&p.tm_k, &k_full[st],
                                     smem + C::OFF_K + st * C::K_BYTES + ch * C::KCHUNK + lane * p.box_rows * C::RB, ch * 64, cy, cz);
            __syncwarp();
            ++it;
        }
        // never leave with copies in flight
        volatile int no_abort = 0;
        for (uint32_t i = it > C::NST ? it - C::NST : 0u; i < it; ++i)
            wait_bar_warp(&k_full[i % C::NST], (i / C::NST) & 1, &no_abort, p.err, true);
        for (uint32_t i = units > C::QB ? units - C::QB : 0u; i < units; ++i)
            wait_bar_warp(&q_full[i % C::QB], (i / C::QB) & 1, &no_abort, p.err, true);
    } else if (warp == 1) {
        // ---------------------------------------------------------------- S^T = K Q^T
        const bool leader = ptx::elect_one();
        const uint32_t sQ = ptx::smem_u32(smem + C::OFF_Q), sK = ptx::smem_u32(smem + C::OFF_K);
        const uint64_t desc = ptx::smem_desc(0, 16, 8 * C::RB, C::SWZ);  // K (A) and Q (B): K-major
        const uint32_t idesc = ptx::idesc_bf16_f32(kWeighKeys, n16, false, false);
        constexpr int KPC = C::RB / 32;  // 16-element steps per column chunk
        WeighWalk walk(p, *plan);
        uint32_t it = 0, units = 0;
        int have = -1;
        bool ok = true;
        while (ok && walk.next()) {
            if (walk.unit != have) {
                if (have >= 0 && leader) ptx::mma_commit(&q_empty[(units - 1) % C::QB]);
                __syncwarp();
                ok = wait_stage_warp(&q_full[units % C::QB], (units / C::QB) & 1, abort_flag, p.err);
                ++units;
                have = walk.unit;
            }
            const uint32_t st = it % C::NST, sb = it & 1;
            ok = ok && wait_stage_warp(&s_free[sb], ((it >> 1) & 1) ^ 1, abort_flag, p.err) &&
                 wait_stage_warp(&k_full[st], (it / C::NST) & 1, abort_flag, p.err);
            if (!ok) break;
            ptx::tc_fence_after();
            if (leader) {
                const uint32_t q = sQ + ((units - 1) % C::QB) * C::Q_BYTES, k = sK + st * C::K_BYTES;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    ptx::mma_ss(tmem + sb * N, desc | ((k + (ks / KPC) * C::KCHUNK + (ks % KPC) * 32) >> 4),
                                desc | ((q + (ks / KPC) * C::QCHUNK + (ks % KPC) * 32) >> 4), idesc, ks > 0 ? 1u : 0u);
                ptx::mma_commit(&k_empty[st]);
                ptx::mma_commit(&s_full[sb]);
            }
            __syncwarp();
            ++it;
        }
        // tensor memory is released when this warp's products and every epilogue thread are done
        if (leader) ptx::mma_commit(drain);
        __syncwarp();
        volatile int no_abort = 0;
        wait_bar_warp(drain, 0, &no_abort, p.err, true);
        wait_bar_warp(done, 0, &no_abort, p.err, true);
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::TMEM_COLS);
    } else if (warp >= 4) {
        // ---------------------------------------------------------------- thread = key: sums over the columns
        // Warpgroup g takes every other tile; every warp has its own copy of the normalisers.
        const int g = (warp - 4) >> 2, w = warp & 3, key = 32 * w + lane;
        float* lse2 = reinterpret_cast<float*>(smem + C::OFF_LSE) + (warp - 4) * N;
        WeighWalk walk(p, *plan);
        // The tile ahead: its weight and its table entry are on their way while this one's scores are waited
        // for.  at < 0: no row of this thread's.
        int unit_n = -1;
        long long at_n = -1;
        float before_n = 0.f;
        int entry_n = 0;
        auto ahead = [&](int skip) {
            bool more = true;
            for (int i = 0; i <= skip && more; ++i) more = walk.next();
            at_n = -1;
            if (!more) return false;
            unit_n = walk.unit;
            const int j = walk.t * kWeighKeys + key;
            if (j < walk.P) {
                at_n = static_cast<long long>(unit_n) * cap + j;
                before_n = __ldcg(p.weight + at_n);
                int in_page;
                entry_n = p.pages.entry(walk.b, j, in_page);
            }
            return true;
        };
        int have = -1;
        bool more = ahead(g);
        for (uint32_t use = 0; more; ++use) {
            const int unit = unit_n;
            const long long at = at_n;
            const float before = before_n;
            const int entry = entry_n;
            more = ahead(1);
            if (unit != have) {
                have = unit;
                __syncwarp();  // the last unit's values have been read
                // -infinity: the column adds nothing, whatever its scores are -- a row that saw nothing (its query may be
                // anything, NaN included), and the columns past the last row, which hold another unit's query, or none,
                // or (past n16) old scores
                for (int c = lane; c < (n16 + 31) / 32 * 32; c += 32)
                    lse2[c] = c < p.n ? __ldcg(p.lse + static_cast<long long>(have) * p.rows + p.row0 + c) * 1.4426950408889634f : -INFINITY;
                __syncwarp();
            }
            if (!wait_stage_warp(&s_full[g], use & 1, abort_flag, p.err)) break;
            ptx::tc_fence_after();
            float sum = 0.f;
            for (int c0 = 0; c0 < n16; c0 += 32) {
                uint32_t raw[32];
                const uint32_t ta = tmem + g * N + (static_cast<uint32_t>(32 * w) << 16) + c0;
                ptx::tmem_ld32(ta, raw);
                ptx::tmem_wait_ld();
                ptx::reg_fence<32>(raw);
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float z = lse2[c0 + c], e = ptx::ex2(__uint_as_float(raw[c]) * p.scale_log2 - z);
                    part[c & 3] += z == -INFINITY ? 0.f : e;
                }
                sum += (part[0] + part[1]) + (part[2] + part[3]);
            }
            ptx::tc_fence_before();
            mbar_arrive_warp(&s_free[g], lane);
            if (at >= 0) p.weight_out[at] = before + (p.pages.page(entry) >= 0 ? sum : 0.f);
        }
        ptx::tc_fence_before();
        mbar_arrive_warp(done, lane);
    }
}

}  // namespace e2d2
