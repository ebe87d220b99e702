// paged_attn_tc.cuh -- the paged sampling step at d = 128, on the 5th-generation tensor cores.
//
// As paged_attn.cuh, but with the products taken transposed and their accumulators in tensor memory:
//
//     S^T  = K Q^T           M = 128 keys (lanes),  N columns = query rows,                  K = d
//     O^T += V^T [P^T | R^T] M = d = 128 (lanes),   2 N columns = probabilities, remainders, K = keys
//
// P and R are the two bf16 that hold a probability to 16 bits and more: the remainders are N more columns of the same
// product, added to the others' when the unit ends.  A tile's softmax is that of 128 threads for every 16 columns
// (thread = key) and the tensor cores work beside it.  HBM bounds it up to 32 query rows per head: 32 single tokens over up
// to 8192 rows take 93 us (5.7 TB/s, 87 % of the copy rate), 32 blocks of 16 tokens over 2048 rows with 32 query rows 51 us
// (5.4 TB/s).  With 64 (4 blocks over up to 32768 rows) the softmax's chain of waits per tile does, and follows the SM's
// clock: 118 us, 4.4 TB/s, as calls one after the other, 103 us in stretches too short to draw the clock down.  Short
// calls are a chain of latencies: one token over 500 rows takes 9.3 us.
//
// A column's running maximum is shared by its warpgroup's 128 keys: each tile the threads vote whether any key beats
// any of their columns' by more than 2^8, and only then are they reduced and O^T rescaled.  It is held negated and in
// the exponent's units, so that one multiply-add gives both the vote's and the exponential's argument.  Warp 0 loads Q and K, warp 2 loads V,
// warp 1 issues S^T (two buffers: the next tile's is computed during this one's softmax), warp 3 issues O^T.  The rings
// run ahead across units.  The cut of the work over blocks, the partial slots and the join are paged_attn.cuh's.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "fmha_keyrow_sm100.cuh"
#include "paged_attn.cuh"

namespace e2d2 {

constexpr int kTcKeys = 128;      // keys of a tile
constexpr int kTcMinKeys = 384;   // keys per block that the split aims for

template <int N_>
struct TcCfg {
    static constexpr int N = N_, D = 128;
    static constexpr int NH = 16;                     // columns per softmax warpgroup
    static constexpr int WGS = N / NH, SOFT = 128 * WGS;  // warpgroups, their threads
    static constexpr int THREADS = 128 + SOFT;        // and four control warps
    // 640 threads start with 96 registers each: 128 x 64 and 512 x 104 are the same 61440 (without: 112 us for 105)
    static constexpr bool SPLIT_REGS = N == 64;
    static constexpr int KV = kTcKeys * D * 2;        // K (or V) of a tile: two column halves of 128-byte rows
    static constexpr int HALF = kTcKeys * 128;
    static constexpr int Q_BYTES = N * D * 2;
    static constexpr int P_CHUNKS = (2 * N + 63) / 64;  // 64-column chunks of [P^T | R^T]
    static constexpr int P_BYTES = P_CHUNKS * HALF;
    static constexpr int NK = N == 64 ? 2 : 3, NV = 2;  // ring stages; [P^T | R^T] is double-buffered
    static constexpr uint32_t TMEM_COLS = 4 * N;      // S^T at 0 and N, O^T at 2 N
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = OFF_Q + Q_BYTES;
    static constexpr int OFF_K = OFF_P + 2 * P_BYTES;
    static constexpr int OFF_V = OFF_K + NK * KV;
    static constexpr int OFF_BAR = OFF_V + NV * KV;
    // q_full, q_empty, k_full[NK], k_empty[NK], v_full[NV], v_empty[NV], s_full[2], s_free[2], p_full[2], pv_done[2],
    // o_free, s_drain, pv_drain, done
    static constexpr int NBAR = 2 + 2 * NK + 2 * NV + 8 + 4;
    static constexpr int OFF_CMAX = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;  // float [WGS][2 parity][4 warps][NH]
    static constexpr int OFF_LRED = OFF_CMAX + WGS * 2 * 4 * NH * 4;      // float [WGS][4 warps][NH]
    static constexpr int OFF_MISC = OFF_LRED + WGS * 4 * NH * 4;          // holder, abort, broadcast
    static constexpr int OFF_PLAN = OFF_MISC + 16;
    static constexpr int OFF_INV = OFF_PLAN + 32;                         // float [N]: 1 / sum of a column
    static constexpr int ALLOC = OFF_INV + N * 4 + 1024;                  // + alignment slack
    static_assert(ALLOC <= 232448 && TMEM_COLS <= 512, "shared and tensor memory");
};

// a * b + c and a + b of pairs of floats, each pair one instruction.
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %6};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1) {
    asm("{\n\t.reg .b64 a, d;\n\t"
        "mov.b64 d, {%0, %1};\n\tmov.b64 a, {%2, %3};\n\t"
        "add.rn.f32x2 d, d, a;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1));
}

// Named barrier of n threads that also says whether any of them brought true.
__device__ __forceinline__ bool barrier_any(uint32_t id, uint32_t n, bool mine) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(any)
        : "r"(mine ? 1u : 0u), "r"(id), "r"(n)
        : "memory");
    return any != 0;
}

template <int N>
__global__ void __launch_bounds__(TcCfg<N>::THREADS, 1) paged_attn_tc_kernel(const __grid_constant__ PagedAttnParams p) {
    using C = TcCfg<N>;
    constexpr int NH = C::NH, D = C::D;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* q_empty = q_full + 1;
    uint64_t* k_full = q_empty + 1;
    uint64_t* k_empty = k_full + C::NK;
    uint64_t* v_full = k_empty + C::NK;
    uint64_t* v_empty = v_full + C::NV;
    uint64_t* s_full = v_empty + C::NV;
    uint64_t* s_free = s_full + 2;
    uint64_t* p_full = s_free + 2;
    uint64_t* pv_done = p_full + 2;
    uint64_t* o_free = pv_done + 2;
    uint64_t* s_drain = o_free + 1;
    uint64_t* pv_drain = s_drain + 1;
    uint64_t* done = pv_drain + 1;
    uint32_t* holder = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    volatile int* bcast = abort_flag + 1;

    ptx::griddep_launch_dependents();
    if (threadIdx.x == 0) {
        ptx::mbar_init(q_full, 1);
        ptx::mbar_init(q_empty, 1);
        for (int i = 0; i < C::NK; ++i) ptx::mbar_init(&k_full[i], 1), ptx::mbar_init(&k_empty[i], 1);
        for (int i = 0; i < C::NV; ++i) ptx::mbar_init(&v_full[i], 1), ptx::mbar_init(&v_empty[i], 1);
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&s_full[i], 1), ptx::mbar_init(&s_free[i], 4 * C::WGS);
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&p_full[i], 4 * C::WGS), ptx::mbar_init(&pv_done[i], 1);
        ptx::mbar_init(o_free, 4 * C::WGS);
        ptx::mbar_init(s_drain, 1);
        ptx::mbar_init(pv_drain, 1);
        ptx::mbar_init(done, 4 * C::WGS);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(holder, C::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    bool delayed = false;
    if (warp == 0 || warp == 2) {
        if (lane == 0) {
            ptx::tma_prefetch_desc(warp == 0 ? &p.tm_k : &p.tm_v);
            ptx::tma_prefetch_desc(warp == 0 ? &p.tm_k1 : &p.tm_v1);
            if (warp == 0) ptx::tma_prefetch_desc(&p.tm_q);
        }
        delayed = producer_delay_set();
    }
    ptx::griddep_wait();  // inputs are read after the previous kernel on the stream has finished
    PagedPlan* plan = reinterpret_cast<PagedPlan*>(smem + C::OFF_PLAN);
    if (warp == 0) paged_plan<kTcKeys, kTcMinKeys>(p, plan);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *holder;
    const int Hkv = p.pages.kv_heads;
    PagedWalk<kTcKeys, N> walk(p, *plan);  // an idle block's has no units: its roles fall through
    // rows of tile c of the unit at hand, and whether it is the own block's
    auto tile_rows = [&](int c, bool& is_own) {
        is_own = c < walk.n_own;
        return (is_own ? walk.own_rows - c * kTcKeys : walk.P - (c - walk.n_own) * kTcKeys);
    };

    if (warp == 0 || warp == 2) {
        // ---------------------------------------------------------------- loads: warp 0 Q and K, warp 2 V
        if constexpr (C::SPLIT_REGS) ptx::setmaxnreg_dec<64>();
        if (delayed) test_producer_delay();
        const bool is_k = warp == 0;
        const int NS = is_k ? C::NK : C::NV;
        uint64_t* full = is_k ? k_full : v_full;
        uint64_t* empty = is_k ? k_empty : v_empty;
        uint8_t* ring = smem + (is_k ? C::OFF_K : C::OFF_V);
        uint32_t it = 0, units = 0;
        bool ok = true;
        while (ok && walk.next()) {
            if (walk.n == 0) continue;
            if (is_k) {
                ok = wait_stage_warp(q_empty, (units & 1) ^ 1, abort_flag, p.err);
                if (!ok) break;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(q_full, C::Q_BYTES);
                    tma_load_q(&p.tm_q, q_full, smem + C::OFF_Q, static_cast<int>(walk.row0));
                }
                __syncwarp();
            }
            ++units;
            // lane j: box j of a tile, its table entry on its way a tile ahead
            auto look_up = [&](int i, int& y, int& e) {
                y = -1;
                e = 0;
                const int c = walk.c0 + i;
                if (i >= walk.n) return;
                const int box = c < walk.n_own ? p.own_box : p.box_rows, in = lane * box;
                const int r = (c < walk.n_own ? c : c - walk.n_own) * kTcKeys + in;
                if (in >= kTcKeys || r >= (c < walk.n_own ? walk.own_rows : walk.P)) return;
                y = r;
                if (c >= walk.n_own) e = p.pages.entry(walk.b, r, y);
            };
            int y_nxt, e_nxt;
            look_up(0, y_nxt, e_nxt);
            for (int i = 0; i < walk.n; ++i) {
                const int y = y_nxt, e = e_nxt;
                look_up(i + 1, y_nxt, e_nxt);
                const bool is_own = walk.c0 + i < walk.n_own;
                const int box = is_own ? p.own_box : p.box_rows;
                int z = walk.b * Hkv + walk.h;
                if (y >= 0 && !is_own && p.pages.table != nullptr) {
                    const int pg = p.pages.page(e);
                    z = pg < 0 ? p.pages.num_pages * Hkv : pg * Hkv + walk.h;  // past the pool: zeros
                }
                const uint32_t st = it % NS;
                ok = wait_stage_warp(&empty[st], ((it / NS) & 1) ^ 1, abort_flag, p.err);
                if (!ok) break;
                const int boxes = __popc(__ballot_sync(0xffffffffu, y >= 0));
                if (lane == 0) ptx::mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(boxes) * box * D * 2);
                __syncwarp();
                if (y >= 0) {
                    const CUtensorMap* map = is_k ? (is_own ? &p.tm_k1 : &p.tm_k) : (is_own ? &p.tm_v1 : &p.tm_v);
                    uint8_t* dst = ring + st * C::KV + lane * box * 128;
                    ptx::tma_load_3d(map, &full[st], dst, 0, y, z);
                    ptx::tma_load_3d(map, &full[st], dst + C::HALF, 64, y, z);
                }
                __syncwarp();
                ++it;
            }
        }
        // never leave with copies in flight
        volatile int no_abort = 0;
        for (uint32_t i = it > static_cast<uint32_t>(NS) ? it - NS : 0u; i < it; ++i)
            wait_bar_warp(&full[i % NS], (i / NS) & 1, &no_abort, p.err, true);
        if (is_k && units > 0) wait_bar_warp(q_full, (units - 1) & 1, &no_abort, p.err, true);
    } else if (warp == 1) {
        // ---------------------------------------------------------------- S^T = K Q^T
        if constexpr (C::SPLIT_REGS) ptx::setmaxnreg_dec<64>();
        const bool leader = ptx::elect_one();
        const uint32_t sQ = ptx::smem_u32(smem + C::OFF_Q), sK = ptx::smem_u32(smem + C::OFF_K);
        const uint64_t desc = ptx::smem_desc(0, 16, 1024, 2u);  // K (A) and Q (B): K-major, 128-byte swizzle
        constexpr uint32_t idesc = ptx::idesc_bf16_f32(kTcKeys, N, false, false);
        uint32_t it = 0, units = 0;
        bool ok = true;
        while (ok && walk.next()) {
            if (walk.n == 0) continue;
            ok = wait_stage_warp(q_full, units & 1, abort_flag, p.err);
            ++units;
            for (int i = 0; i < walk.n && ok; ++i) {
                const uint32_t st = it % C::NK, sb = it & 1;
                ok = wait_stage_warp(&s_free[sb], ((it >> 1) & 1) ^ 1, abort_flag, p.err) &&
                     wait_stage_warp(&k_full[st], (it / C::NK) & 1, abort_flag, p.err);
                if (!ok) break;
                ptx::tc_fence_after();
                if (leader) {
                    const uint32_t k = sK + st * C::KV;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        ptx::mma_ss(tmem + sb * N, desc | ((k + (ks / 4) * C::HALF + (ks % 4) * 32) >> 4),
                                    desc | ((sQ + (ks / 4) * (N * 128) + (ks % 4) * 32) >> 4), idesc, ks > 0 ? 1u : 0u);
                    ptx::mma_commit(&k_empty[st]);
                    ptx::mma_commit(&s_full[sb]);
                    if (i == walk.n - 1) ptx::mma_commit(q_empty);
                }
                __syncwarp();
                ++it;
            }
        }
        // tensor memory is released when both issuers' products and every softmax thread are done
        if (leader) ptx::mma_commit(s_drain);
        __syncwarp();
        volatile int no_abort = 0;
        wait_bar_warp(s_drain, 0, &no_abort, p.err, true);
        wait_bar_warp(pv_drain, 0, &no_abort, p.err, true);
        wait_bar_warp(done, 0, &no_abort, p.err, true);
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::TMEM_COLS);
    } else if (warp == 3) {
        // ---------------------------------------------------------------- O^T += V^T [P^T | R^T]
        if constexpr (C::SPLIT_REGS) ptx::setmaxnreg_dec<64>();
        const bool leader = ptx::elect_one();
        const uint32_t sP = ptx::smem_u32(smem + C::OFF_P), sV = ptx::smem_u32(smem + C::OFF_V);
        const uint64_t desc = ptx::smem_desc(0, C::HALF, 1024, 2u);  // both MN-major: V^T (d contiguous), P^T (columns)
        constexpr uint32_t idesc = ptx::idesc_bf16_f32(D, 2 * N, true, true);
        uint32_t it = 0, units = 0;
        bool ok = true;
        while (ok && walk.next()) {
            if (walk.n == 0) continue;
            for (int i = 0; i < walk.n && ok; ++i) {
                const uint32_t st = it % C::NV;
                const uint32_t sb = it & 1;
                ok = wait_stage_warp(&p_full[sb], (it >> 1) & 1, abort_flag, p.err) &&
                     (i > 0 || wait_stage_warp(o_free, (units & 1) ^ 1, abort_flag, p.err)) &&
                     wait_stage_warp(&v_full[st], (it / C::NV) & 1, abort_flag, p.err);
                if (!ok) break;
                ptx::tc_fence_after();
                bool is_own;
                const int steps = (min(kTcKeys, tile_rows(walk.c0 + i, is_own)) + 15) / 16;
                if (leader) {
                    const uint32_t v = sV + st * C::KV, pr = sP + sb * C::P_BYTES;
                    for (int ks = 0; ks < steps; ++ks)
                        ptx::mma_ss(tmem + 2 * N, desc | ((v + ks * 16 * 128) >> 4), desc | ((pr + ks * 16 * 128) >> 4), idesc,
                                    i > 0 || ks > 0 ? 1u : 0u);
                    ptx::mma_commit(&v_empty[st]);
                    ptx::mma_commit(&pv_done[sb]);
                }
                __syncwarp();
                ++it;
            }
            ++units;
        }
        if (leader) ptx::mma_commit(pv_drain);
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax: thread = key lane, warpgroup = columns
        // Waits never break the loops: every warp takes every named barrier.
        if constexpr (C::SPLIT_REGS) ptx::setmaxnreg_inc<104>();
        const int g = (warp - 4) >> 2, w = warp & 3, key = 32 * w + lane, tid = threadIdx.x - 128;
        const uint32_t lane_off = static_cast<uint32_t>(32 * w) << 16;
        const uint32_t o_tmem = tmem + lane_off + 2 * N + g * NH;  // these columns' probabilities; remainders N columns on
        float* cmax = reinterpret_cast<float*>(smem + C::OFF_CMAX) + g * 2 * 4 * NH;
        float* lred = reinterpret_cast<float*>(smem + C::OFF_LRED) + g * 4 * NH;
        uint8_t* sP = smem + C::OFF_P;
        constexpr float kNone = 3.0e38f;  // -(maximum) of a column without keys: finite, so that -inf scores give 0
        uint32_t tc = 0;
        while (walk.next()) {
            float neg_m[NH], l_part[NH];
#pragma unroll
            for (int j = 0; j < NH; ++j) neg_m[j] = kNone, l_part[j] = 0.f;
            // the table's entry for this thread's key, on its way a tile ahead
            auto entry_of = [&](int i) {
                const int c = walk.c0 + i, j = (c - walk.n_own) * kTcKeys + key;
                int in_page;
                return i < walk.n && c >= walk.n_own && j < walk.P ? p.pages.entry(walk.b, j, in_page) : 0;
            };
            int e_nxt = entry_of(0);
            for (int i = 0; i < walk.n; ++i, ++tc) {
                const uint32_t sb = tc & 1;
                const int e = e_nxt;
                e_nxt = entry_of(i + 1);
                bool is_own;
                const int valid = tile_rows(walk.c0 + i, is_own);
                bool key_ok = key < valid;
                if (key_ok && !is_own) key_ok = p.pages.page(e) >= 0;
                wait_stage_warp(&s_full[sb], (tc >> 1) & 1, abort_flag, p.err);
                ptx::tc_fence_after();
                // x = a key's scores, then the exponents scale x - m.  The scores are read again where a maximum moves.
                float x[NH];
                auto scores = [&]() {
                    uint32_t raw[NH];
                    ptx::tmem_ld16(tmem + sb * N + lane_off + g * NH, raw);
                    ptx::tmem_wait_ld();
                    ptx::reg_fence<NH>(raw);
#pragma unroll
                    for (int j = 0; j < NH; ++j) x[j] = __uint_as_float(raw[j]);
                };
                auto exponents = [&]() {
#pragma unroll
                    for (int j = 0; j < NH; j += 2)
                        fma2(x[j], x[j + 1], x[j], x[j + 1], p.scale_log2, neg_m[j], neg_m[j + 1]);
                };
                auto mask = [&]() {
                    if (!__all_sync(0xffffffffu, key_ok)) {
                        if (!key_ok)
#pragma unroll
                            for (int j = 0; j < NH; ++j) x[j] = -INFINITY;
                    }
                };
                scores();
                exponents();
                mask();
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < NH; j += 2) top = ptx::fmax3(top, x[j], x[j + 1]);
                if (barrier_any(1 + g, 128, top > kRescaleThreshold)) {
                    // new maxima, of every column whose keys reach past the old one
                    scores();
                    mask();
                    float tmp[NH];
#pragma unroll
                    for (int j = 0; j < NH; ++j) tmp[j] = x[j] * p.scale_log2;
                    const float mine = warp_columns_reduce<NH>(tmp, lane, [](float a, float b) { return fmaxf(a, b); });
                    float* cm = cmax + sb * 4 * NH;
                    if ((lane % (32 / NH)) == 0) cm[w * NH + lane / (32 / NH)] = mine;
                    ptx::named_barrier_sync(1 + g, 128);
                    if (i > 0) {  // O^T holds every product up to the last tile's once that one has landed
                        wait_stage_warp(&pv_done[sb ^ 1], ((tc - 1) >> 1) & 1, abort_flag, p.err);
                        ptx::tc_fence_after();
                    }
#pragma unroll
                    for (int c8 = 0; c8 < NH; c8 += 8) {
                        float fac[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int j = c8 + k;
                            const float tm = fmaxf(fmaxf(cm[j], cm[NH + j]), fmaxf(cm[2 * NH + j], cm[3 * NH + j]));
                            const float nm = fminf(neg_m[j], tm == -INFINITY ? kNone : -tm);
                            fac[k] = ptx::ex2(nm - neg_m[j]);
                            neg_m[j] = nm;
                            l_part[j] *= fac[k];
                        }
                        if (i > 0) {
#pragma unroll
                            for (int part = 0; part < 2; ++part) {  // probabilities, remainders
                                uint32_t o[8];
                                ptx::tmem_ld8(o_tmem + part * N + c8, o);
                                ptx::tmem_wait_ld();
                                ptx::reg_fence<8>(o);
#pragma unroll
                                for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fac[k]);
                                ptx::tmem_st8(o_tmem + part * N + c8, o);
                            }
                        }
                    }
                    if (i > 0) ptx::tmem_wait_st();
                    exponents();
                    mask();
                }
                ptx::tc_fence_before();
                mbar_arrive_warp(&s_free[sb], lane);  // the next S^T product may overwrite the buffer
                // this key's row of [P^T | R^T]: exp2(x - m) as bf16 and bf16 remainder
                uint32_t hi[NH / 2], lo[NH / 2];
#pragma unroll
                for (int j = 0; j < NH; j += 2) {
                    const float e0 = ptx::ex2(x[j]), e1 = ptx::ex2(x[j + 1]);
                    add2(l_part[j], l_part[j + 1], e0, e1);
                    const uint32_t h2 = ptx::pack_bf16x2(e0, e1);
                    hi[j / 2] = h2;
                    float r0, r1;  // e - value, exact
                    fma2(r0, r1, __uint_as_float(h2 << 16), __uint_as_float(h2 & 0xffff0000u), -1.f, e0, e1);
                    lo[j / 2] = ptx::pack_bf16x2(r0, r1);
                }
                // the buffer was read by the product of the tile before last
                wait_stage_warp(&pv_done[sb], ((tc >> 1) & 1) ^ 1, abort_flag, p.err);
                uint8_t* pr = sP + sb * C::P_BYTES;
#pragma unroll
                for (int u = 0; u < NH / 8; ++u) {
                    const int uh = g * (NH / 8) + u, ul = N / 8 + uh;  // 16-byte units of the row
                    *reinterpret_cast<uint4*>(pr + uh / 8 * C::HALF + swz_rows<128>(key, uh % 8)) =
                        make_uint4(hi[4 * u], hi[4 * u + 1], hi[4 * u + 2], hi[4 * u + 3]);
                    *reinterpret_cast<uint4*>(pr + ul / 8 * C::HALF + swz_rows<128>(key, ul % 8)) =
                        make_uint4(lo[4 * u], lo[4 * u + 1], lo[4 * u + 2], lo[4 * u + 3]);
                }
                if (g == 0 && !is_own && valid < kTcKeys && (valid & 15) != 0) {
                    // Rows past the length in the last 16 keys that the product takes may hold anything (NaN
                    // included), and meet zero probabilities: they become zero.
                    const uint32_t st = tc % C::NV;
                    wait_stage_warp(&v_full[st], (tc / C::NV) & 1, abort_flag, p.err);
                    if (key >= valid && key < ((valid + 15) & ~15)) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint4* dst = reinterpret_cast<uint4*>(smem + C::OFF_V + st * C::KV + half * C::HALF + key * 128);
#pragma unroll
                            for (int u = 0; u < 8; ++u) dst[u] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                }
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
                mbar_arrive_warp(&p_full[sb], lane);
            }
            // ---- the unit's end: column sums over the keys, O^T out of tensor memory
            const bool whole = walk.whole;
            const int rows_here = walk.rows_here;
            const int c_first = whole ? 0 : walk.first_block();
            float* slot = whole ? nullptr : walk.slot(blockIdx.x, c_first);
            float* inv_l = reinterpret_cast<float*>(smem + C::OFF_INV) + g * NH;
            if (walk.n > 0) {
                const float mine = warp_columns_reduce<NH>(l_part, lane, [](float a, float b) { return a + b; });
                if ((lane % (32 / NH)) == 0) lred[w * NH + lane / (32 / NH)] = mine;
                ptx::named_barrier_sync(1 + g, 128);
            }
            if (w == 0 && lane < NH) {
                // lane = column: its sum, maximum, normaliser
                const float l = walk.n > 0 ? (lred[lane] + lred[NH + lane]) + (lred[2 * NH + lane] + lred[3 * NH + lane]) : 0.f;
                float nm = neg_m[0];
#pragma unroll
                for (int j = 1; j < NH; ++j) nm = lane == j ? neg_m[j] : nm;
                const int col = g * NH + lane;
                if (whole) {
                    // (a unit without keys writes zeros and leaves the last unit's values to their readers)
                    if (walk.n > 0) inv_l[lane] = l == 0.f ? 0.f : 1.f / l;
                    if (p.lse != nullptr && col < rows_here)
                        p.lse[walk.row0 + col] = l == 0.f ? -INFINITY : (log2f(l) - nm) * 0.69314718055994531f;
                } else if (col < rows_here) {
                    __stcg(slot + p.rows_cap * D + col, l == 0.f ? -INFINITY : -nm);
                    __stcg(slot + p.rows_cap * D + p.rows_cap + col, l);
                }
            }
            if (walk.n > 0) {
                wait_stage_warp(&pv_done[(tc - 1) & 1], ((tc - 1) >> 1) & 1, abort_flag, p.err);
                ptx::tc_fence_after();
            }
            if (whole) ptx::named_barrier_sync(1 + g, 128);  // inv_l is written
            const int cols = min(NH, rows_here - g * NH);    // rows of this warpgroup's columns
            __nv_bfloat16* out = p.out + (walk.row0 + g * NH) * D + key;
            float* part = whole ? nullptr : slot + g * NH * D + key;
#pragma unroll 1
            for (int c8 = 0; c8 < NH; c8 += 8) {
                uint32_t oh[8], ol[8];
                if (walk.n > 0) {
                    ptx::tmem_ld8(o_tmem + c8, oh);
                    ptx::tmem_ld8(o_tmem + N + c8, ol);
                    ptx::tmem_wait_ld();
                    ptx::reg_fence<8>(oh);
                    ptx::reg_fence<8>(ol);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) oh[k] = ol[k] = 0u;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    // an infinite value's products: infinite with the probabilities, anything with the remainders
                    const float hi = __uint_as_float(oh[k]), o = fabsf(hi) == INFINITY ? hi : hi + __uint_as_float(ol[k]);
                    if (whole) {
                        if (c8 + k < cols) out[(c8 + k) * D] = __float2bfloat16_rn(walk.n > 0 ? o * inv_l[c8 + k] : 0.f);
                    } else if (c8 + k < cols) {
                        __stcg(part + (c8 + k) * D, o);
                    }
                }
            }
            if (walk.n > 0) {
                ptx::tc_fence_before();
                mbar_arrive_warp(o_free, lane);
            }
            if (!whole) {
                // publish; the last block of the unit joins all of them
                ptx::named_barrier_sync(1 + C::WGS, C::SOFT);
                const int c_last = walk.last_block();
                if (tid == 0) {
                    __threadfence();
                    const int ticket = atomicAdd(&p.tickets[c_first], 1);
                    const int last = ticket == c_last - c_first;
                    if (last) p.tickets[c_first] = 0;
                    *bcast = last;
                }
                ptx::named_barrier_sync(1 + C::WGS, C::SOFT);
                const bool join = *bcast != 0;
                ptx::named_barrier_sync(1 + C::WGS, C::SOFT);  // read before the next unit's is written
                if (join) {
                    __threadfence();
                    // few rows: many parts in flight (token, 18 parts: 14.8 against 17.8 us for the call); many rows: many rows
                    // (64 rows, 5 parts: 105 against 108 us)
                    join_parts<D, 4 * C::WGS, N == 16 ? 1 : 4, N == 16 ? 8 : 2>(p, walk.slot(c_first, c_first), walk.slot(c_first + 1, c_first), c_last - c_first + 1,
                                           walk.row0, rows_here, warp - 4, lane);
                }
            }
        }
        ptx::tc_fence_before();
        mbar_arrive_warp(done, lane);
    }
}

}  // namespace e2d2
