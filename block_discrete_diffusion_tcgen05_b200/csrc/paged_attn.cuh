// paged_attn.cuh -- the sampling step over a paged KV cache.
//
//   x_ij = scale q_i . k_j,  lse_i = log sum_j exp(x_ij),  out_i = sum_j exp(x_ij - lse_i) v_j
//
// for the S query rows of a block (one row: a single new token) and every query head, over the P[b] cached
// rows of the entry and, when given, the block's own S rows.
//
// A kv head's keys are read once for the G S query rows that share it (a unit of work; 128 rows at most, more
// rows are more units), so a call is bound by HBM until some 64 rows share a head.  Everything is arranged for
// bytes in flight: a warp owns a ring of shared-memory stages of CK keys (K and V, one TMA box per 16 rows, so
// a page of any multiple of 16 rows is a whole number of boxes), refills a stage itself the moment it has
// used it, and runs the online softmax of its own keys with its own running maximum, without a word to the
// other warps before the unit ends.  Two blocks of four warps per SM: one streams while the other joins its
// warps' results.
//
// The products use mma.sync with the query rows on the 16-row side: with 1 to 32 rows a tensor-memory
// accumulator would be almost empty, and the scores would have to travel TMEM -> registers -> shared memory
// between the two products, where here they stay in the registers that the first product leaves them in.  The
// probabilities enter the second product as the sum of two bf16 (value and remainder): held to 16 bits and
// more, they add nothing to the rounding of the output, for tensor-core time that the loads hide.
//
// The chunks of all units form one stream that is cut evenly over the blocks (lengths are read on the device,
// so any mix of lengths is balanced); a unit that several blocks share is joined by the last of them, from
// fp32 partial results in the workspace, in the blocks' order.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "kv_paged.cuh"

namespace e2d2 {

constexpr int kPagedThreads = 128;
constexpr int kPagedMaxCtas = 320;   // workspace sizing: tickets and partial slots
constexpr int kPagedStats = 8192;    // row statistics of the parts of a unit that are joined at a time
constexpr int kPagedMinChunks = 16;  // chunks per block that the split aims for

struct alignas(64) PagedAttnParams {
    CUtensorMap tm_k, tm_v;    // pools: 3D {D, page_rows, num_pages * Hkv}, boxes of 16 rows
    CUtensorMap tm_k1, tm_v1;  // own block: 3D {D, S, B * Hkv}
    PageView pages;
    const uint4* q;            // [B][Hq][S][D] bf16
    const int* P_dev;
    __nv_bfloat16* out;        // [B][Hq][S][D]
    float* lse;                // [B][Hq][S] or null
    int* tickets;              // one per block
    float* partial;            // two slots per block
    unsigned int* err;
    int batch, q_heads, group, S;
    int own;                   // the block's own rows take part
    int rows;                  // G * S packed query rows per kv head
    int qtiles;                // query tiles per kv head
    int rows_cap, slot_floats; // rows of a partial slot, its floats
    float scale_log2;          // softmax scale * log2(e)
};

template <int D_, int MT_, int RW_>
struct PagedCfg {
    static constexpr int D = D_;
    static constexpr int MT = MT_;             // 16-row tiles per warp
    static constexpr int RW = RW_;             // warps that share a ring, each with its own rows
    static constexpr int KG = 4 / RW;          // rings: warps (or groups) with their own keys
    static constexpr int ROWS = 16 * MT * RW;  // query rows of a unit
    static constexpr int CK = D == 128 ? 16 : 32;           // keys of a stage
    static constexpr int SUB = CK / 16;                     // 16-row boxes of it
    static constexpr int RB = D * 2 < 128 ? D * 2 : 128;    // bytes per row of one column chunk
    static constexpr int NCH = D * 2 / RB;
    static constexpr int BOX = 16 * RB;
    static constexpr int SUBB = BOX * NCH;                  // K (or V) of 16 keys
    static constexpr int KB = SUB * SUBB;
    static constexpr int STAGE = 2 * KB;
    static constexpr int Q_BYTES = ROWS * D * 2;
    static constexpr int RING = (110 * 1024 - 4096 - Q_BYTES) / (KG * STAGE) * (KG * STAGE);
    static constexpr int NST = RING / (KG * STAGE) < 12 ? RING / (KG * STAGE) : 12;
    static constexpr int RSTRIDE = D + 8;                   // floats per row of the join buffer (in the ring)
    static constexpr int JOIN = KG * ROWS * RSTRIDE * 4;
    static constexpr int PRE = (kPagedMaxBatch + 1) * 8;    // prefix table of the schedule (in the ring)
    static constexpr int USED = KG * NST * STAGE;
    static constexpr int STATS = 2 * kPagedStats * 4;       // the join's row statistics (in the ring)
    static constexpr int max2(int a, int b) { return a > b ? a : b; }
    static constexpr int RING_BYTES = (max2(max2(USED, STATS), max2(JOIN, PRE)) + 1023) / 1024 * 1024;
    static constexpr int OFF_RING = 0;
    static constexpr int OFF_Q = RING_BYTES;
    static constexpr int OFF_BAR = OFF_Q + Q_BYTES;          // full[KG][NST], empty[KG][NST]
    static constexpr int OFF_BAD = OFF_BAR + 2 * KG * NST * 8;  // int [KG][NST]: boxes of no page
    static constexpr int OFF_STAT = (OFF_BAD + KG * NST * 4 + 15) / 16 * 16;  // float m[KG][ROWS], l[KG][ROWS]
    static constexpr int OFF_MISC = OFF_STAT + 2 * KG * ROWS * 4;
    static constexpr int BYTES = OFF_MISC + 64;
    static constexpr int ALLOC = (BYTES + 1023) / 1024 * 1024 + 1024;
    static_assert(NST >= 2 && NST * SUB <= 32 && ALLOC <= 113 * 1024, "two blocks per SM");
    static constexpr bool QREG = MT == 1;      // query fragments stay in registers
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte unit u of row r in a block of 16 rows of D bf16, as the swizzled TMA boxes (one per
// column chunk of RB bytes) leave it.
template <int D>
__device__ __forceinline__ uint32_t box_offset(int r, int u) {
    constexpr int RB = D * 2 < 128 ? D * 2 : 128, UPC = RB / 16;
    const int x = RB == 128 ? (r & 7) : ((r >> 1) & 3);
    return static_cast<uint32_t>((u / UPC) * (16 * RB) + r * RB + (((u % UPC) ^ x) << 4));
}

// Chunks of a unit's keys: the own block's, then the cached rows'.
__device__ __forceinline__ int paged_chunks(int P, int own_rows, int ck) {
    return (own_rows + ck - 1) / ck + (P + ck - 1) / ck;
}

template <int D, int MT, int RW>
__global__ void __launch_bounds__(kPagedThreads, 2) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
    using C = PagedCfg<D, MT, RW>;
    constexpr int CK = C::CK, SUB = C::SUB, KG = C::KG, NST = C::NST, ROWS = C::ROWS;
    constexpr int NT = D / 8;  // 8-column tiles of an output row
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int kg = warp / RW, rw = warp % RW;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + kg * NST;
    uint64_t* empty = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + KG * NST + kg * NST;
    volatile int* bad = reinterpret_cast<volatile int*>(smem + C::OFF_BAD) + kg * NST;
    float* stat_m = reinterpret_cast<float*>(smem + C::OFF_STAT);
    float* stat_l = stat_m + KG * ROWS;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
    volatile int* bcast = abort_flag + 1;
    long long* scan_sums = reinterpret_cast<long long*>(smem + C::OFF_MISC + 16);  // [4]

    ptx::griddep_launch_dependents();
    if (tid == 0) {
        uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
        for (int i = 0; i < KG * NST; ++i) {
            ptx::mbar_init(bars + i, 1);
            ptx::mbar_init(bars + KG * NST + i, RW);
        }
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::tma_prefetch_desc(&p.tm_k);
        ptx::tma_prefetch_desc(&p.tm_v);
    }
    ptx::griddep_wait();  // lengths, table and rows are read after the previous kernel on the stream

    // ---- schedule: pre[b] = stream chunks before entry b, then this block's range and the entry it starts in
    const int Hkv = p.pages.kv_heads, cap = p.pages.capacity();
    const int upe = Hkv * p.qtiles;  // units per entry
    const int own_rows = p.own ? p.S : 0;
    const int n_own = (own_rows + CK - 1) / CK;
    long long* pre = reinterpret_cast<long long*>(smem + C::OFF_RING);
    long long total, pos, end, ent_beg;
    int b, sgrid;
    {
        total = stream_prefix<kPagedThreads>(p.batch, pre, scan_sums, [&](int i) {
            return static_cast<long long>(upe) * max(1, paged_chunks(ragged_clamp(__ldcg(p.P_dev + i), cap), own_rows, CK));
        });
        // as many blocks as keep about kPagedMinChunks chunks each, one per unit at least, at most the grid
        long long g = total / kPagedMinChunks;
        const long long units = static_cast<long long>(p.batch) * upe;
        if (g < units) g = units;
        if (g > gridDim.x) g = gridDim.x;
        sgrid = static_cast<int>(g);  // total >= units, so every block has a chunk
        if (static_cast<int>(blockIdx.x) >= sgrid) return;
        pos = range_begin(blockIdx.x, total, sgrid);
        end = range_begin(blockIdx.x + 1, total, sgrid);
        b = stream_entry(pre, p.batch, pos);
        ent_beg = pre[b];
    }

    const uint32_t ring = ptx::smem_u32(smem + C::OFF_RING) + kg * NST * C::STAGE;
    const uint32_t sq = ptx::smem_u32(smem + C::OFF_Q) + rw * MT * (16 * D * 2);
    const int g8 = lane >> 2, t4 = lane & 3;
    // ldmatrix lane addresses: matrix lane / 8, row lane % 8
    const int l7 = lane & 7, mat = lane >> 3;
    const int rk = l7 + (mat >> 1) * 8, uk = mat & 1;  // K: keys 0-7, 8-15 of two 16-byte units
    const int rv = l7 + (mat & 1) * 8, uv = mat >> 1;  // V (transposed) and Q
    uint32_t it = 0;  // stages used by this ring so far
    bool ok = true;
    test_producer_delay();

    while (pos < end) {
        // ---- the unit: entry b, kv head h, query tile qt; its chunks [c0, c1) fall to this block
        const int P = ragged_clamp(__ldcg(p.P_dev + b), cap);
        const int real = paged_chunks(P, own_rows, CK);
        const int Cu = max(1, real);
        const int u_in = static_cast<int>((pos - ent_beg) / Cu);
        const long long ubeg = ent_beg + static_cast<long long>(u_in) * Cu;
        const int h = u_in / p.qtiles, qt = u_in - h * p.qtiles;
        const int c0 = static_cast<int>(pos - ubeg);
        const int c1 = static_cast<int>((end < ubeg + Cu ? end : ubeg + Cu) - ubeg);
        const bool whole = c0 == 0 && c1 == Cu;
        const int own_z = b * Hkv + h;
        const int rows_here = min(ROWS, p.rows - qt * ROWS);
        const long long row0 = (static_cast<long long>(b) * p.q_heads + static_cast<long long>(h) * p.group) * p.S +
                               static_cast<long long>(qt) * ROWS;
        const int n_my = max(0, (min(c1, real) - c0 - kg + KG - 1) / KG);  // chunks c0 + kg, c0 + kg + KG, ...

        // The ring's generic writes (schedule table, or the join of the last unit) are over and visible to
        // the copies that follow.
        ptx::fence_proxy_async_smem();
        __syncthreads();

        // Boxes of this ring in their order: box q = sub-block q % SUB of chunk q / SUB.  Lane j looks up box
        // 32 n + j: (row inside the page, pool index); cur covers the boxes being issued, nxt the 32 after.
        auto look_up = [&](int q, int& y, int& z) {
            const int i = q / SUB, c = c0 + kg + i * KG;
            y = -1;  // nothing to load
            z = own_z;
            if (i >= n_my) return;
            if (c < n_own) {
                const int r = c * CK + (q % SUB) * 16;
                if (r < own_rows) y = r;
                return;
            }
            const int r = (c - n_own) * CK + (q % SUB) * 16;
            if (r >= P) return;
            y = r;
            if (p.pages.table != nullptr) {
                const int pg = p.pages.page_of(b, r);
                y = r % p.pages.page_rows;
                z = pg < 0 ? p.pages.num_pages * Hkv : pg * Hkv + h;  // past the pool: zeros are loaded
            }
        };
        int y_cur = -1, z_cur = 0, y_nxt = -1, z_nxt = 0;
        auto issue = [&](int i) {  // chunk i of this ring into its stage; the whole warp calls it, i < n_my
            const int q0 = i * SUB;
            if (q0 % 32 == 0) {
                if (i == 0) look_up(lane, y_cur, z_cur);
                else y_cur = y_nxt, z_cur = z_nxt;
                look_up(q0 + 32 + lane, y_nxt, z_nxt);
            }
            int y[SUB], z[SUB], n = 0, bad_bits = 0;
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
                y[s] = __shfl_sync(0xffffffffu, y_cur, (q0 + s) % 32);
                z[s] = __shfl_sync(0xffffffffu, z_cur, (q0 + s) % 32);
                n += y[s] >= 0;
            }
            const int c = c0 + kg + i * KG;
            const bool is_own = c < n_own;
            if (!is_own)
#pragma unroll
                for (int s = 0; s < SUB; ++s) bad_bits |= (y[s] >= 0 && z[s] == p.pages.num_pages * Hkv) ? 1 << s : 0;
            const uint32_t st = (it + i) % NST;
            if (lane == 0) {
                bad[st] = bad_bits;  // released to the readers by the arrival
                ptx::mbar_arrive_expect_tx(&full[st], n * 2 * C::SUBB);
                uint8_t* dst = smem + C::OFF_RING + (kg * NST + st) * C::STAGE;
                const CUtensorMap* mk = is_own ? &p.tm_k1 : &p.tm_k;
                const CUtensorMap* mv = is_own ? &p.tm_v1 : &p.tm_v;
#pragma unroll
                for (int s = 0; s < SUB; ++s) {
                    if (y[s] < 0) continue;
#pragma unroll
                    for (int ch = 0; ch < C::NCH; ++ch) {
                        ptx::tma_load_3d(mk, &full[st], dst + s * C::SUBB + ch * C::BOX, ch * 64, y[s], z[s]);
                        ptx::tma_load_3d(mv, &full[st], dst + C::KB + s * C::SUBB + ch * C::BOX, ch * 64, y[s], z[s]);
                    }
                }
            }
            __syncwarp();
        };
        int issued = 0;
        if (rw == 0)
            for (; issued < n_my && issued < NST; ++issued) issue(issued);

        // ---- the unit's query rows, rows past the last one zero
        for (int i = tid; i < ROWS * (D / 8); i += kPagedThreads) {
            const int r = i / (D / 8), u = i % (D / 8);
            const uint4 x = r < rows_here ? __ldcg(p.q + (row0 + r) * (D / 8) + u) : make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(smem + C::OFF_Q + (r / 16) * (16 * D * 2) + box_offset<D>(r % 16, u)) = x;
        }
        __syncthreads();
        uint32_t qf[C::QREG ? D / 16 : 1][4];
        if constexpr (C::QREG)
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) ldsm4(sq + box_offset<D>(rv, 2 * ks + uv), qf[ks]);

        float o[MT][NT][4], m[MT][2], l[MT][2];
#pragma unroll
        for (int a = 0; a < MT; ++a) {
            m[a][0] = m[a][1] = -INFINITY;
            l[a][0] = l[a][1] = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) o[a][n][0] = o[a][n][1] = o[a][n][2] = o[a][n][3] = 0.f;
        }

        for (int i = 0; i < n_my && ok; ++i) {
            const uint32_t st = (it + i) % NST;
            ok = wait_bar_warp(&full[st], ((it + i) / NST) & 1, abort_flag, p.err);
            if (!ok) break;
            const uint32_t sk = ring + st * C::STAGE, sv = sk + C::KB;
            const int c = c0 + kg + i * KG;
            const int valid = c < n_own ? own_rows - c * CK : P - (c - n_own) * CK;  // keys of the chunk in range
            const int bad_bits = bad[st];

            // S = Q K^T
            float s[MT][2 * SUB][4];
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int n = 0; n < 2 * SUB; ++n) s[a][n][0] = s[a][n][1] = s[a][n][2] = s[a][n][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t qa[MT][4];
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    if constexpr (C::QREG) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) qa[a][e] = qf[ks][e];
                    } else {
                        ldsm4(sq + a * (16 * D * 2) + box_offset<D>(rv, 2 * ks + uv), qa[a]);
                    }
                }
#pragma unroll
                for (int sb = 0; sb < SUB; ++sb) {
                    uint32_t kb[4];
                    ldsm4(sk + sb * C::SUBB + box_offset<D>(rk, 2 * ks + uk), kb);
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
                        mma_16816(s[a][2 * sb], qa[a], kb[0], kb[1]);
                        mma_16816(s[a][2 * sb + 1], qa[a], kb[2], kb[3]);
                    }
                }
            }
            // Keys past the end, and those of boxes that no page backs, get no weight; their V rows (anything,
            // NaN included) must not meet the product with a zero probability, so they become zero.
            const bool cut = valid < CK || bad_bits != 0;
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int n = 0; n < 2 * SUB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[a][n][e] *= p.scale_log2;
            if (cut) {
#pragma unroll
                for (int n = 0; n < 2 * SUB; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = n * 8 + 2 * t4 + (e & 1);
                        if (key >= valid || ((bad_bits >> (n / 2)) & 1))
#pragma unroll
                            for (int a = 0; a < MT; ++a) s[a][n][e] = -INFINITY;
                    }
                for (int x = lane; x < CK * (D / 8); x += 32) {
                    const int key = x / (D / 8), u = x % (D / 8);
                    if (key >= valid)
                        *reinterpret_cast<uint4*>(smem + C::OFF_RING + (kg * NST + st) * C::STAGE + C::KB +
                                                  (key / 16) * C::SUBB + box_offset<D>(key % 16, u)) = make_uint4(0u, 0u, 0u, 0u);
                }
                __syncwarp();
                ptx::fence_proxy_async_smem();  // before the stage is loaded again
            }
            // Running maximum, moved only when a score beats it by 2^8 (sums and outputs stay far inside fp32)
            uint32_t moved = 0;
            float mx[MT][2];
#pragma unroll
            for (int a = 0; a < MT; ++a)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float x = s[a][0][2 * r];
#pragma unroll
                    for (int n = 0; n < 2 * SUB; ++n) x = fmaxf(x, fmaxf(s[a][n][2 * r], s[a][n][2 * r + 1]));
                    mx[a][r] = x;
                    moved |= x > m[a][r] + kRescaleThreshold;
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float x = mx[a][r];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                        const float mn = fmaxf(m[a][r], x);
                        const float f = m[a][r] == -INFINITY ? 0.f : ptx::ex2(m[a][r] - mn);
                        m[a][r] = mn;
                        l[a][r] *= f;
#pragma unroll
                        for (int n = 0; n < NT; ++n) o[a][n][2 * r] *= f, o[a][n][2 * r + 1] *= f;
                    }
            }
            // P = exp2(S - m), as bf16 plus bf16 remainder: the first product's accumulators are the second's
            // A fragments
            uint32_t ph[MT][SUB][4], pl[MT][SUB][4];
#pragma unroll
            for (int a = 0; a < MT; ++a) {
                const float m0 = m[a][0] == -INFINITY ? 0.f : m[a][0], m1 = m[a][1] == -INFINITY ? 0.f : m[a][1];
#pragma unroll
                for (int sb = 0; sb < SUB; ++sb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // fragment register e: rows g (e even), g + 8; keys 2t, 2t + 8
                        const float* x = &s[a][2 * sb + (e >> 1)][2 * (e & 1)];
                        const float mm = (e & 1) ? m1 : m0;
                        const float p0 = ptx::ex2(x[0] - mm), p1 = ptx::ex2(x[1] - mm);
                        l[a][e & 1] += p0 + p1;
                        const uint32_t hi = ptx::pack_bf16x2(p0, p1);
                        ph[a][sb][e] = hi;
                        pl[a][sb][e] = ptx::pack_bf16x2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
                    }
            }
            // O += P V
#pragma unroll
            for (int sb = 0; sb < SUB; ++sb)
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t vb[4];
                    ldsm4t(sv + sb * C::SUBB + box_offset<D>(rv, 2 * j + uv), vb);
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
                        mma_16816(o[a][2 * j], ph[a][sb], vb[0], vb[1]);
                        mma_16816(o[a][2 * j + 1], ph[a][sb], vb[2], vb[3]);
                        mma_16816(o[a][2 * j], pl[a][sb], vb[0], vb[1]);
                        mma_16816(o[a][2 * j + 1], pl[a][sb], vb[2], vb[3]);
                    }
                }
            // The stage is free: load the chunk NST further on.
            __syncwarp();
            if constexpr (RW > 1) {
                if (lane == 0) ptx::mbar_arrive(&empty[st]);
                if (rw == 0 && issued < n_my) {
                    ok = wait_bar_warp(&empty[st], ((it + i) / NST) & 1, abort_flag, p.err);
                    if (ok) issue(issued++);
                }
            } else {
                if (issued < n_my) issue(issued++);
            }
        }
        if (!ok && rw == 0) {
            // never leave with copies in flight
            volatile int no_abort = 0;
            for (int i = issued > NST ? issued - NST : 0; i < issued; ++i)
                wait_bar_warp(&full[(it + i) % NST], ((it + i) / NST) & 1, &no_abort, p.err, true);
        }
        it += n_my;

        // ---- join the rings: row statistics, then the scaled sums through shared memory
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = l[a][r];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                l[a][r] = x;
                if (t4 == 0) stat_m[kg * ROWS + (rw * MT + a) * 16 + g8 + 8 * r] = m[a][r];
            }
        __syncthreads();  // every ring is drained, every maximum written
        if (*abort_flag) return;
        float* join = reinterpret_cast<float*>(smem + C::OFF_RING);
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = (rw * MT + a) * 16 + g8 + 8 * r;
                float mt = stat_m[row];
#pragma unroll
                for (int k = 1; k < KG; ++k) mt = fmaxf(mt, stat_m[k * ROWS + row]);
                const float f = m[a][r] == -INFINITY ? 0.f : ptx::ex2(m[a][r] - mt);
                if (t4 == 0) stat_l[kg * ROWS + row] = l[a][r] * f;
                float* dst = join + (kg * ROWS + row) * C::RSTRIDE + 2 * t4;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[a][n][2 * r] * f, o[a][n][2 * r + 1] * f);
            }
        __syncthreads();
        const int c_first = whole ? 0 : owner_cta(ubeg, total, sgrid);
        const int c_last = whole ? 0 : owner_cta(ubeg + Cu - 1, total, sgrid);
        // A block's first unit takes its slot 2 c when it began before or at the block's range, a unit that begins
        // inside the range takes 2 c + 1: of a unit's blocks only the first can be the latter.
        const bool inside = !whole && range_begin(c_first, total, sgrid) < ubeg;
        auto slot_of = [&](int c) {
            return p.partial + static_cast<size_t>(2 * c + (c == c_first && inside)) * p.slot_floats;
        };
        float* slot = whole ? nullptr : slot_of(blockIdx.x);
        for (int i = tid; i < rows_here * (D / 4); i += kPagedThreads) {
            const int row = i / (D / 4), q4 = i % (D / 4);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float lt = 0.f;
#pragma unroll
            for (int k = 0; k < KG; ++k) {
                const float4 x = *reinterpret_cast<const float4*>(join + (k * ROWS + row) * C::RSTRIDE + q4 * 4);
                acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
                lt += stat_l[k * ROWS + row];
            }
            float mt = stat_m[row];
#pragma unroll
            for (int k = 1; k < KG; ++k) mt = fmaxf(mt, stat_m[k * ROWS + row]);
            if (whole) {
                const float inv = lt > 0.f ? 1.f / lt : 0.f;  // a row that sees nothing: zeros, lse = -inf
                uint2 w;
                w.x = ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
                w.y = ptx::pack_bf16x2(acc.z * inv, acc.w * inv);
                *reinterpret_cast<uint2*>(p.out + (row0 + row) * D + q4 * 4) = w;
                if (q4 == 0 && p.lse != nullptr)
                    p.lse[row0 + row] = lt > 0.f ? (mt + log2f(lt)) * 0.69314718055994531f : -INFINITY;
            } else {
                *reinterpret_cast<float4*>(slot + row * D + q4 * 4) = acc;
                if (q4 == 0) {
                    slot[p.rows_cap * D + row] = mt;
                    slot[p.rows_cap * D + p.rows_cap + row] = lt;
                }
            }
        }
        if (!whole) {
            // publish; the last block of the unit joins all of them
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                const int ticket = atomicAdd(&p.tickets[c_first], 1);
                const int last = ticket == c_last - c_first;
                if (last) p.tickets[c_first] = 0;
                *bcast = last;
            }
            __syncthreads();
            if (*bcast) {
                __threadfence();
                // The ring is free: row statistics of a few rows at a time in shared memory, [part][row], then
                // the parts' rows from L2 with several loads in flight per thread.
                const int parts = c_last - c_first + 1;
                const int rp = min(rows_here, kPagedStats / parts);
                float* fm = join;            // maxima, then factors 2^(m - max)
                float* fl = join + kPagedStats;     // sums
                for (int r0 = 0; r0 < rows_here; r0 += rp) {
                    const int nr = min(rp, rows_here - r0);
                    for (int i = tid; i < parts * nr; i += kPagedThreads) {
                        const int c = i / nr, row = i - c * nr;
                        const float* st = slot_of(c_first + c) + p.rows_cap * D + r0 + row;
                        fm[i] = __ldcg(st);
                        fl[i] = __ldcg(st + p.rows_cap);
                    }
                    __syncthreads();
                    // eight lanes per row
                    for (int i = tid; i < (nr * 8 + 31) / 32 * 32; i += kPagedThreads) {
                        const int row = i >> 3, part = i & 7;
                        float mt = -INFINITY, lt = 0.f;
                        if (row < nr)
                            for (int c = part; c < parts; c += 8) mt = fmaxf(mt, fm[c * nr + row]);
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
                        if (row < nr)
                            for (int c = part; c < parts; c += 8) {
                                const float mc = fm[c * nr + row];
                                const float f = mc == -INFINITY ? 0.f : ptx::ex2(mc - mt);
                                fm[c * nr + row] = f;
                                lt += fl[c * nr + row] * f;
                            }
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
                        if (row < nr && part == 0) {
                            fl[row] = lt > 0.f ? 1.f / lt : 0.f;  // part 0's sum of this row: read above, by these lanes only
                            if (p.lse != nullptr)
                                p.lse[row0 + r0 + row] = lt > 0.f ? (mt + log2f(lt)) * 0.69314718055994531f : -INFINITY;
                        }
                    }
                    __syncthreads();
                    constexpr int IT = 4;
                    const int items = nr * (D / 4);
                    for (int i0 = tid; i0 < items; i0 += IT * kPagedThreads) {
                        float4 acc[IT];
#pragma unroll
                        for (int k = 0; k < IT; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                        for (int c = 0; c < parts; ++c) {
                            const float4* sl = reinterpret_cast<const float4*>(slot_of(c_first + c)) + r0 * (D / 4);
#pragma unroll
                            for (int k = 0; k < IT; ++k) {
                                const int i = i0 + k * kPagedThreads;
                                if (i >= items) continue;
                                const float4 x = __ldcg(sl + i);
                                const float f = fm[c * nr + i / (D / 4)];
                                acc[k].x += x.x * f, acc[k].y += x.y * f, acc[k].z += x.z * f, acc[k].w += x.w * f;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < IT; ++k) {
                            const int i = i0 + k * kPagedThreads;
                            if (i >= items) continue;
                            const float inv = fl[i / (D / 4)];
                            uint2 w;
                            w.x = ptx::pack_bf16x2(acc[k].x * inv, acc[k].y * inv);
                            w.y = ptx::pack_bf16x2(acc[k].z * inv, acc[k].w * inv);
                            *reinterpret_cast<uint2*>(p.out + (row0 + r0) * D + i * 4) = w;
                        }
                    }
                    __syncthreads();
                }
            }
        }
        pos = ubeg + c1;
        if (u_in + 1 == upe && c1 == Cu) {
            ent_beg += static_cast<long long>(upe) * Cu;
            ++b;
        }
        __syncthreads();  // the join buffer has been read: the ring may be loaded again
    }
}

}  // namespace e2d2
