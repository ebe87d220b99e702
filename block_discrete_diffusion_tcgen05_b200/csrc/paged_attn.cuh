// paged_attn.cuh -- the sampling step over a paged KV cache: the cut of the work over blocks and the join of their
// parts, for every head size, and the kernel for head sizes 32 and 64 (128: paged_attn_tc.cuh).
//
//   x_ij = scale q_i . k_j,  lse_i = log sum_j exp(x_ij),  out_i = sum_j exp(x_ij - lse_i) v_j
//
// for the S query rows of a block (one row: a single new token) and every query head, over the P[b] cached
// rows of the entry and, when given, the block's own S rows.
//
// A kv head's keys are read once for the G S query rows that share it (a unit of work; 64 rows at most, more
// rows are more units), so a call is bound by HBM until some 64 rows share a head.  Everything is arranged for
// bytes in flight.  A block is one warp that loads and four that compute; three blocks share an SM, so one streams
// while another starts or joins.  The loader fills a ring of stages, K and V, in boxes of as many rows as pages
// allow (16 at least: a page of any multiple of 16 rows is a whole number of boxes; issuing copies is what bounds a
// loader, about a hundred clocks each), and its lanes look up the pages of the next stages ahead of time.  A
// consumer warp takes 32 keys of every stage and 16 query rows, and runs the online softmax of its own keys with its own
// running maximum, without a word to the others before the unit ends.
//
// The products use mma.sync with the query rows on the 16-row side: head sizes 32 and 64 do not fill the 128 lanes that
// V^T P^T takes in tensor memory, and the scores stay in the registers that the first product leaves them in, where
// the second one wants them.  The probabilities enter the second product as the sum of two bf16 (value and remainder):
// held to 16 bits, they add nothing to the rounding of the output, for tensor-core time that the loads hide.  32 single
// tokens over up to 8192 rows take 48 us at d = 64 (85 % of the copy rate); with 64 query rows per head (4 blocks over
// 4000..8000 rows, d = 64) the warps wait for the products' latencies and one another: 39 us, a fifth of the copy rate.
// At d = 128 this kernel took 92.9 us for 32 single tokens over up to 8192 rows (89 % of the copy rate) against 95.2 us
// of the tensor-memory kernel, but 11.8 against 9.5 us for one token over 500 rows, and 68 against 52 us and 198
// against 109 us for blocks of 32 and 64 query rows.
//
// The stages of all units form one stream that is cut evenly over the blocks (lengths are read on the device,
// so any mix of lengths is balanced); where lengths differ a unit takes kPagedUnitStages empty places ahead of its
// stages, so that a block with many short units does not take as many stages as the others on top.  A unit that
// several blocks share is joined by the last of them, from fp32 partial results in the workspace, in the blocks'
// order.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "kv_paged.cuh"

namespace e2d2 {

constexpr int kPagedMaxCtas = 480;  // workspace sizing: tickets and partial slots
constexpr int kPagedMaxRows = 64;   // query rows of a unit
constexpr int kPagedUnitStages = 4; // what beginning and joining a unit costs, in stages, where lengths differ
constexpr int kPagedMinKeys = 256;  // keys per block that the split aims for

struct alignas(64) PagedAttnParams {
    CUtensorMap tm_k, tm_v;    // pools: 3D {D, page_rows, num_pages * Hkv}, boxes of box_rows
    CUtensorMap tm_k1, tm_v1;  // own block: 3D {D, S, B * Hkv}, boxes of own_box
    CUtensorMap tm_q;          // queries: rows of [B * Hq * S][D], every column of a unit's rows in a box
    PageView pages;
    const int* P_dev;
    __nv_bfloat16* out;        // [B][Hq][S][D]
    float* lse;                // [B][Hq][S] or null
    int* tickets;              // one per block
    float* partial;            // two slots per block
    unsigned int* err;
    int batch, q_heads, group, S;
    int box_rows, own_box;
    int own;                   // the block's own rows take part
    int rows;                  // G * S packed query rows per kv head
    int qtiles;                // query tiles per kv head
    int rows_cap, slot_floats; // rows of a partial slot, its floats
    float scale_log2;          // softmax scale * log2(e)
};

// RW: 16-row groups of query rows (1, 2, 4).  The four consumer warps are 4 / RW slices of a stage's keys times RW
// row groups.  Every warp uses every stage, so none can take one phase of a stage's barrier for another.  Three
// blocks of five warps leave 128 registers per thread.
template <int D_, int RW_>
struct PagedCfg {
    static constexpr int D = D_, RW = RW_;
    static_assert(D == 32 || D == 64, "one column chunk per row");
    static constexpr int CTAS = 3;                          // blocks per SM
    static constexpr int WARPS = 4;                         // consumer warps
    static constexpr int THREADS = 32 * (WARPS + 1);
    static constexpr int SLICES = WARPS / RW;
    static constexpr int ROWS = 16 * RW;                    // query rows of a unit
    static constexpr int SK = 32;                           // keys of a slice
    static constexpr int SUB = SK / 16;
    static constexpr int KEYS = SK * SLICES;                // keys of a stage
    static constexpr int RB = D * 2;                        // bytes per row
    static constexpr int KB = KEYS * RB;
    static constexpr int STAGE = 2 * KB;
    static constexpr int RING = (RW <= 2 ? 64 : 48) * 1024;
    static constexpr int NST = RING / STAGE;
    static constexpr int Q_BYTES = ROWS * RB;
    static constexpr int RSTRIDE = D + 8;                   // floats per row of the join buffer (in the ring)
    static_assert(SLICES * ROWS * RSTRIDE * 4 <= RING, "the ring holds the join");
    static constexpr int OFF_RING = 0;
    static constexpr int OFF_Q = RING;
    static constexpr int OFF_BAR = OFF_Q + Q_BYTES;         // full[NST], empty[NST], q_full
    static constexpr int OFF_BAD = OFF_BAR + (2 * NST + 1) * 8;   // int [NST]: groups of 16 keys that no page backs
    static constexpr int OFF_STAT = (OFF_BAD + NST * 4 + 15) / 16 * 16;  // float m[SLICES][ROWS], l[SLICES][ROWS]
    static constexpr int OFF_MISC = OFF_STAT + 2 * SLICES * ROWS * 4;    // abort, broadcast
    static constexpr int OFF_PLAN = OFF_MISC + 16;
    static constexpr int ALLOC = OFF_PLAN + 32 + 1024;      // + alignment slack
    static_assert(NST >= 2 && CTAS * (ALLOC + 1024) <= 228 * 1024, "shared memory");
};

// A box of query rows from row y on, all columns (the row's halves of 128 bytes are a dimension of the map).
__device__ __forceinline__ void tma_load_q(const CUtensorMap* map, uint64_t* bar, void* dst, int y) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %3, %3}], [%2];" ::"r"(ptx::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(0), "r"(y)
        : "memory");
}

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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte unit u of row r in a tile of rows of D bf16, as the swizzled TMA boxes leave it.
template <int D>
__device__ __forceinline__ uint32_t tile_offset(int r, int u) {
    const int x = D == 64 ? (r & 7) : ((r >> 1) & 3);
    return static_cast<uint32_t>(r * D * 2 + ((u ^ x) << 4));
}

// Stages of a unit's keys: the own block's, then the cached rows'.
__device__ __forceinline__ int paged_stages(int P, int own_rows, int keys) {
    return (own_rows + keys - 1) / keys + (P + keys - 1) / keys;
}

// A stream of `total` stages (below 2^31, the host sees to it) cut over `parts` blocks: block c takes
// [begin(c), begin(c + 1)), begin(c) = floor(c total / parts).
struct StreamCut {
    unsigned total, q, r;
    int parts;
    __device__ StreamCut(unsigned t, int n) : total(t), q(t / n), r(t % n), parts(n) {}
    __device__ unsigned begin(unsigned c) const { return c * q + (c * r) / parts; }  // c r < parts^2
    // begin(c) <= x, without the division
    __device__ bool begins_by(int c, unsigned x) const {
        return static_cast<unsigned long long>(c) * total < (x + 1ull) * parts;
    }
    // The block that holds stage x: an estimate (off by less than one block), then its neighbours.
    __device__ int owner(unsigned x) const {
        int c = static_cast<int>(__fdividef(static_cast<float>(x), static_cast<float>(total)) * parts);
        c = max(0, min(c, parts - 1));
        while (!begins_by(c, x)) --c;
        while (c + 1 < parts && begins_by(c + 1, x)) ++c;
        return c;
    }
};

// Blocks that a call's stream is cut over: as many as keep about min_stages stages each, one per unit at least, at
// most the grid.  Units of equal length are cut at their ends -- into equal parts each, or so many whole units per
// block -- if that leaves no more than a fifth of the blocks idle: a block whose range meets the ends of two units
// publishes and joins twice.
__device__ __forceinline__ int paged_parts(unsigned total, unsigned units, bool equal, unsigned grid, int min_stages) {
    const unsigned want = max(total / min_stages, units);
    if (want < grid) return equal ? want - want % units : want;
    if (!equal) return grid;
    const unsigned per = (units + grid - 1) / grid;  // whole units per block, where there are more units than blocks
    const unsigned aligned = units <= grid ? grid - grid % units : (units % per == 0 ? units / per : 0);
    return 5 * aligned >= 4 * grid ? aligned : grid;
}

// Four columns of an output row from their weighted sum and the sum of the weights.
__device__ __forceinline__ void write_row4(const PagedAttnParams& p, long long at, int D, int q4, float l, const float4& acc) {
    const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing: zeros (NaN stays NaN)
    uint2 w;
    w.x = ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
    w.y = ptx::pack_bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(p.out + at * D + q4 * 4) = w;
}

// The last block of a shared unit: joins its parts, in the blocks' order, and writes the rows.  The first part's
// slot, then one every two slots from `rest`.  D / 4 lanes per row, four columns each, IT rows and AT parts in flight;
// lane k of a row's lanes takes part k's maximum and sum.  No shared memory, no barrier.
template <int D, int WARPS, int IT, int AT>
__device__ __forceinline__ void join_parts(const PagedAttnParams& p, const float* first, const float* rest, int parts,
                                           long long row0, int rows, int warp, int lane) {
    constexpr int LPR = D / 4, RPW = 32 / LPR;
    const int li = lane % LPR;
    auto part = [&](int k) { return k == 0 ? first : rest + static_cast<size_t>(2 * (k - 1)) * p.slot_floats; };
#pragma unroll 1
    for (int base = warp * RPW; base < rows; base += WARPS * RPW * IT) {
        int row[IT];
        float mt[IT], lt[IT];
        float4 acc[IT];
#pragma unroll
        for (int y = 0; y < IT; ++y) {
            row[y] = min(base + WARPS * RPW * y + lane / LPR, rows - 1);
            mt[y] = -INFINITY;
            lt[y] = 0.f;
            acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 1
        for (int k0 = 0; k0 < parts; k0 += LPR) {  // as many parts as a row has lanes
            const int np = min(LPR, parts - k0);
            const float* st = part(k0 + min(li, np - 1)) + p.rows_cap * D;
            float f[IT], lc[IT];
            float4 x[AT][IT];
#pragma unroll
            for (int y = 0; y < IT; ++y) {
                f[y] = li < np ? __ldcg(st + row[y]) : -INFINITY;
                lc[y] = __ldcg(st + p.rows_cap + row[y]);
            }
#pragma unroll
            for (int k = 0; k < AT; ++k)
#pragma unroll
                for (int y = 0; y < IT; ++y)
                    x[k][y] = __ldcg(reinterpret_cast<const float4*>(part(k0 + min(k, np - 1)) + row[y] * D) + li);
#pragma unroll
            for (int y = 0; y < IT; ++y) {
                float mn = f[y];
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                mn = fmaxf(mn, mt[y]);
                const float f_old = mt[y] == -INFINITY ? 0.f : ptx::ex2(mt[y] - mn);
                f[y] = f[y] == -INFINITY ? 0.f : ptx::ex2(f[y] - mn);
                float ls = li < np ? lc[y] * f[y] : 0.f;
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
                lt[y] = lt[y] * f_old + ls;
                mt[y] = mn;
                acc[y].x *= f_old, acc[y].y *= f_old, acc[y].z *= f_old, acc[y].w *= f_old;
            }
#pragma unroll 1
            for (int k = 0; k < np; k += AT) {
#pragma unroll
                for (int z = 0; z < AT; ++z)
#pragma unroll
                    for (int y = 0; y < IT; ++y) {
                        const float fk = __shfl_sync(0xffffffffu, f[y], (lane & ~(LPR - 1)) + min(k + z, LPR - 1));
                        if (k + z < np) {
                            acc[y].x += x[z][y].x * fk, acc[y].y += x[z][y].y * fk;
                            acc[y].z += x[z][y].z * fk, acc[y].w += x[z][y].w * fk;
                        }
                    }
                if (k + AT < np)
#pragma unroll
                    for (int z = 0; z < AT; ++z)
#pragma unroll
                        for (int y = 0; y < IT; ++y)
                            x[z][y] = __ldcg(reinterpret_cast<const float4*>(part(k0 + min(k + AT + z, np - 1)) + row[y] * D) + li);
            }
        }
#pragma unroll
        for (int y = 0; y < IT; ++y)
            if (base + WARPS * RPW * y + lane / LPR < rows) {
                write_row4(p, row0 + row[y], D, li, lt[y], acc[y]);
                if (li == 0 && p.lse != nullptr)
                    p.lse[row0 + row[y]] = lt[y] == 0.f ? -INFINITY : (mt[y] + log2f(lt[y])) * 0.69314718055994531f;
            }
    }
}

// A block's place in the stream, worked out by one warp for all (every warp for itself cost more in issue slots).
struct PagedPlan {
    unsigned lead, pos, end, ent_beg, total;
    int parts, b, P;
};

// KEYS: of a stage; MIN_KEYS: that a block of a cut unit should keep.  One warp calls it.
template <int KEYS, int MIN_KEYS>
__device__ __forceinline__ void paged_plan(const PagedAttnParams& p, PagedPlan* out) {
    const int upe = p.pages.kv_heads * p.qtiles, own = p.own ? p.S : 0;
    auto stream = entry_stream(p.P_dev, p.batch, p.pages.capacity(), upe,
                               [own](int rows) { return static_cast<unsigned>(max(1, paged_stages(rows, own, KEYS))); });
    PagedPlan n;
    n.lead = stream.equal ? 0 : kPagedUnitStages;  // empty places ahead of a unit's stages
    stream.lead = n.lead;
    n.total = stream.total + n.lead * p.batch * upe;
    n.parts = paged_parts(n.total, p.batch * upe, stream.equal, gridDim.x, MIN_KEYS / KEYS);
    n.pos = n.end = n.ent_beg = 0;
    n.b = n.P = 0;
    if (static_cast<int>(blockIdx.x) < n.parts) {
        const StreamCut cut(n.total, n.parts);
        n.pos = cut.begin(blockIdx.x);
        n.end = cut.begin(blockIdx.x + 1);
        stream.find(n.pos, n.b, n.ent_beg, n.P);
    }
    if ((threadIdx.x & 31) == 0) *out = n;
}

// The units of a block: its range of the stream, unit by unit.  ROWS: query rows of a unit.  Every thread of a warp
// walks alike.
template <int KEYS, int ROWS>
struct PagedWalk {
    const PagedAttnParams& p;
    int upe, own_rows, n_own;     // units per entry; the own block's rows and stages
    unsigned lead, pos, end, ent_beg, total;
    int parts, next_b, next_P;
    // the unit at hand: entry b with P rows, kv head h; its stages [c0, c0 + n) are this block's
    int b, P, h, c0, n, rows_here;
    long long row0;               // its first row in [B][Hq][S]
    unsigned ubeg, len;           // its first place in the stream, its places
    bool whole;                   // all of it is this block's

    __device__ PagedWalk(const PagedAttnParams& prm, const PagedPlan& n)
        : p(prm), lead(n.lead), pos(n.pos), end(n.end), ent_beg(n.ent_beg), total(n.total), parts(n.parts), next_b(n.b), next_P(n.P) {
        upe = p.pages.kv_heads * p.qtiles;
        own_rows = p.own ? p.S : 0;
        n_own = (own_rows + KEYS - 1) / KEYS;
    }
    __device__ bool idle() const { return static_cast<int>(blockIdx.x) >= parts; }
    __device__ bool next() {
        while (pos < end) {
            b = next_b;
            P = next_P;
            const int real = paged_stages(P, own_rows, KEYS), all = max(1, real);
            len = lead + all;
            const int u_in = (pos - ent_beg) / len;
            ubeg = ent_beg + u_in * len;
            const unsigned past = min(end - ubeg, len);
            h = p.qtiles == 1 ? u_in : u_in / p.qtiles;
            const int qt = u_in - h * p.qtiles;
            c0 = max(static_cast<int>(pos - ubeg - lead), 0);
            const int c1 = max(static_cast<int>(past - lead), 0);
            pos = ubeg + past;
            if (u_in + 1 == upe && past == len) {
                ent_beg += upe * len;
                ++next_b;
                if (pos < end) next_P = ragged_clamp(__ldcg(p.P_dev + next_b), p.pages.capacity());
            }
            if (c0 == c1) continue;  // empty places only
            whole = c0 == 0 && c1 == all;
            n = max(0, min(c1, real) - c0);
            rows_here = min(ROWS, p.rows - qt * ROWS);
            row0 = (static_cast<long long>(b) * p.q_heads + static_cast<long long>(h) * p.group) * p.S +
                   static_cast<long long>(qt) * ROWS;
            return true;
        }
        return false;
    }
    // Blocks that share the unit: the first and the last with one of its stages.
    __device__ int first_block() const { return StreamCut(total, parts).owner(ubeg + lead); }
    __device__ int last_block() const { return StreamCut(total, parts).owner(ubeg + len - 1); }
    // The slot of the unit's block c: a block begins one shared unit at most and goes on with one at most.
    __device__ float* slot(int c, int first) const {
        return p.partial + static_cast<size_t>(2 * c + (c == first)) * p.slot_floats;
    }
};

template <int D, int RW>
__global__ void __launch_bounds__(PagedCfg<D, RW>::THREADS, PagedCfg<D, RW>::CTAS)
    paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
    using C = PagedCfg<D, RW>;
    constexpr int KEYS = C::KEYS, SUB = C::SUB, NST = C::NST, ROWS = C::ROWS, SK = C::SK, SLICES = C::SLICES;
    constexpr int NT = D / 8;                  // 8-column tiles of an output row
    constexpr int NCONS = 32 * C::WARPS;       // consumer threads
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const bool loads = warp == C::WARPS;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + NST;
    uint64_t* q_full = empty + NST;
    volatile int* bad = reinterpret_cast<volatile int*>(smem + C::OFF_BAD);
    float* stat_m = reinterpret_cast<float*>(smem + C::OFF_STAT);
    float* stat_l = stat_m + SLICES * ROWS;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
    volatile int* bcast = abort_flag + 1;

    ptx::griddep_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], C::WARPS);
        }
        ptx::mbar_init(q_full, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (loads && lane == 0) {
        ptx::tma_prefetch_desc(&p.tm_q);
        ptx::tma_prefetch_desc(&p.tm_k);
        ptx::tma_prefetch_desc(&p.tm_v);
    }
    const bool delayed = loads && producer_delay_set();
    ptx::griddep_wait();  // lengths, table and rows are read after the previous kernel on the stream

    PagedPlan* plan = reinterpret_cast<PagedPlan*>(smem + C::OFF_PLAN);
    if (loads) paged_plan<KEYS, kPagedMinKeys>(p, plan);
    __syncthreads();  // the barriers are initialised, the plan is written
    PagedWalk<KEYS, ROWS> walk(p, *plan);
    if (walk.idle()) return;
    if (delayed) test_producer_delay();

    const int rw = warp % RW, slice = warp / RW;
    const uint32_t ring = ptx::smem_u32(smem + C::OFF_RING);
    const int g8 = lane >> 2, t4 = lane & 3;
    // ldmatrix lane addresses: matrix lane / 8, row lane % 8.  K: keys 0-7, 8-15 of two 16-byte units; V
    // (transposed) and Q: rows 0-7, 8-15 of one unit, then of the next.  The swizzle depends on the lane alone; step j
    // (two units) is an XOR of 32 j.
    const int l7 = lane & 7, mat = lane >> 3, key0 = slice * SK;
    const uint32_t ok_ = tile_offset<D>(key0 + l7 + (mat >> 1) * 8, mat & 1);
    const uint32_t ov_ = tile_offset<D>(key0 + l7 + (mat & 1) * 8, mat >> 1);
    const uint32_t oq_ = ptx::smem_u32(smem + C::OFF_Q) + tile_offset<D>(rw * 16 + l7 + (mat & 1) * 8, mat >> 1);
    uint32_t it = 0, n_units = 0;    // stages that went through the ring so far, units

    const int Hkv = p.pages.kv_heads;
    while (walk.next()) {
        const int unit_b = walk.b, unit_P = walk.P, h = walk.h, c0 = walk.c0, n = walk.n, rows_here = walk.rows_here;
        const int n_own = walk.n_own, own_rows = walk.own_rows;
        const bool whole = walk.whole;
        const long long row0 = walk.row0;

        if (loads) {
            // ------------------------------------------------------------ loads
            // The unit's query rows come first, ahead of the stages that would fill the memory pipe.  Rows past the
            // unit's last are other units' (or zeros): no row's result depends on another row.
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(q_full, C::Q_BYTES);
                tma_load_q(&p.tm_q, q_full, smem + C::OFF_Q, static_cast<int>(row0));
            }
            __syncwarp();
            // A batch of 32 look-ups, NB of each stage: cur covers the stages being issued, nxt those after, loaded
            // but not looked at before their turn.
            constexpr int NB = KEYS / 16, SPB = 32 / NB;
            const int z_none = p.pages.num_pages * Hkv;  // past the pool: zeros are loaded
            auto look_up = [&](int i, int& y, int& e) {  // box lane % NB of stage i: row in its page, table entry
                y = -1;
                e = 0;
                const int c = c0 + i;
                if (i >= n) return;
                const int box = c < n_own ? p.own_box : p.box_rows, in = (lane % NB) * box;
                const int r = (c < n_own ? c : c - n_own) * KEYS + in;
                if (in >= KEYS || r >= (c < n_own ? own_rows : unit_P)) return;
                y = r;
                if (c >= n_own) e = p.pages.entry(unit_b, r, y);
            };
            auto pool_index = [&](int i, int y, int e) {
                if (y < 0 || c0 + i < n_own || p.pages.table == nullptr) return unit_b * Hkv + h;
                const int pg = p.pages.page(e);
                return pg < 0 ? z_none : pg * Hkv + h;
            };
            int y_cur = -1, z_cur = 0, y_nxt, e_nxt;
            look_up(lane / NB, y_nxt, e_nxt);
            bool ok = true;
            int i = 0;
            uint32_t st = it % NST, use = it / NST;
            for (; i < n; ++i) {
                const int in_batch = i % SPB;
                if (in_batch == 0) {
                    y_cur = y_nxt;
                    z_cur = pool_index(i + lane / NB, y_nxt, e_nxt);
                    look_up(i + SPB + lane / NB, y_nxt, e_nxt);
                }
                const int y = __shfl_sync(0xffffffffu, y_cur, in_batch * NB + lane % NB);
                const int z = __shfl_sync(0xffffffffu, z_cur, in_batch * NB + lane % NB);
                const bool mine = lane < NB && y >= 0, is_own = c0 + i < n_own;
                const int box = is_own ? p.own_box : p.box_rows;
                const unsigned boxes = __ballot_sync(0xffffffffu, mine);
                const bool none = mine && !is_own && z == z_none;
                unsigned lost = 0;
                if (__any_sync(0xffffffffu, none))
                    lost = __reduce_or_sync(0xffffffffu, none ? ((1u << (box / 16)) - 1u) << (lane * box / 16) : 0u);
                ok = wait_stage_warp(&empty[st], (use & 1) ^ 1, abort_flag, p.err);
                if (!ok) break;
                if (lane == 0) {
                    bad[st] = static_cast<int>(lost);  // released to the readers by the arrival
                    ptx::mbar_arrive_expect_tx(&full[st], __popc(boxes) * static_cast<uint32_t>(box) * (2 * D * 2));
                }
                __syncwarp();
                if (mine) {
                    uint8_t* dst = smem + C::OFF_RING + st * C::STAGE + lane * box * C::RB;
                    ptx::tma_load_3d(is_own ? &p.tm_k1 : &p.tm_k, &full[st], dst, 0, y, z);
                    ptx::tma_load_3d(is_own ? &p.tm_v1 : &p.tm_v, &full[st], dst + C::KB, 0, y, z);
                }
                __syncwarp();
                if (++st == NST) st = 0, ++use;
            }
            // every load has landed before shared memory is used for anything else, timed out or not
            volatile int no_abort = 0;
            for (int k = i > NST ? i - NST : 0; k < i; ++k)
                wait_bar_warp(&full[(it + k) % NST], ((it + k) / NST) & 1, &no_abort, p.err, true);
            wait_bar_warp(q_full, n_units & 1, &no_abort, p.err, true);
        } else {
            // ------------------------------------------------------------ consumers
            const bool q_ok = wait_stage_warp(q_full, n_units & 1, abort_flag, p.err);
            float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
            for (int x = 0; x < NT; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;

            uint32_t st = it % NST, use = it / NST;
            for (int i = 0; i < n && q_ok; ++i) {
                if (!wait_stage_warp(&full[st], use & 1, abort_flag, p.err)) break;
                const int c = c0 + i;
                const bool is_own = c < n_own;
                // keys of this warp's slice that exist (any number, 0 and below for none)
                const int valid = (is_own ? own_rows - c * KEYS : unit_P - (c - n_own) * KEYS) - key0;
                const int lost = (bad[st] >> (slice * SUB)) & ((1 << SUB) - 1);
                if (valid > 0) {
                    const uint32_t sk = ring + st * C::STAGE + ok_, sv = ring + st * C::STAGE + C::KB + ov_;
                    // S = Q K^T, even and odd steps in accumulators of their own (shorter chains)
                    float s[2 * SUB][4], s1[2 * SUB][4];
#pragma unroll
                    for (int x = 0; x < 2 * SUB; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[x][e] = s1[x][e] = 0.f;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        uint32_t qa[4];
                        ldsm4(oq_ ^ (ks * 32), qa);
#pragma unroll
                        for (int sb = 0; sb < SUB; ++sb) {
                            uint32_t kb[4];
                            ldsm4((sk ^ (ks * 32)) + sb * 16 * C::RB, kb);
                            mma_16816((ks & 1) ? s1[2 * sb] : s[2 * sb], qa, kb[0], kb[1]);
                            mma_16816((ks & 1) ? s1[2 * sb + 1] : s[2 * sb + 1], qa, kb[2], kb[3]);
                        }
                    }
#pragma unroll
                    for (int x = 0; x < 2 * SUB; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[x][e] += s1[x][e];
                    // Keys past the end, and those that no page backs, get no weight; their V rows (anything, NaN
                    // included) must not meet the product with a zero probability, so they become zero.
                    if (valid < SK || lost != 0) {
#pragma unroll
                        for (int x = 0; x < 2 * SUB; ++x)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (x * 8 + 2 * t4 + (e & 1) >= valid || ((lost >> (x / 2)) & 1)) s[x][e] = -INFINITY;
                        uint8_t* v0 = smem + C::OFF_RING + st * C::STAGE + C::KB;
                        for (int x = lane; x < SK * (D / 8); x += 32) {
                            const int key = x / (D / 8), u = x % (D / 8);
                            if (key >= valid) *reinterpret_cast<uint4*>(v0 + tile_offset<D>(key0 + key, u)) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        ptx::fence_proxy_async_smem();  // before the stage is loaded again
                        __syncwarp();
                    }
                    // Running maximum (of the raw products), moved only when a score beats it by 2^8: sums and
                    // outputs stay far inside fp32
                    float mx[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        mx[r] = s[0][2 * r];
#pragma unroll
                        for (int x = 0; x < 2 * SUB; ++x) mx[r] = fmaxf(mx[r], fmaxf(s[x][2 * r], s[x][2 * r + 1]));
                    }
                    const bool moved = mx[0] * p.scale_log2 > m[0] + kRescaleThreshold || mx[1] * p.scale_log2 > m[1] + kRescaleThreshold;
                    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float x = mx[r] * p.scale_log2;
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                            const float mn = fmaxf(m[r], x);
                            const float f = m[r] == -INFINITY ? 0.f : ptx::ex2(m[r] - mn);
                            m[r] = mn;
                            l[r] *= f;
#pragma unroll
                            for (int y = 0; y < NT; ++y) o[y][2 * r] *= f, o[y][2 * r + 1] *= f;
                        }
                    }
                    // P = exp2(S - m), as bf16 plus bf16 remainder: the first product's accumulators are the second's A
                    // fragments.  The bf16 is the largest below the probability, so that the remainder has its sign
                    // (at most 2^-7 of it, rounded to within 2^-16): an infinite V row gives infinity, where a remainder
                    // of zero or below gives NaN.
                    const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
                    uint32_t ph[SUB][4], pl[SUB][4];
#pragma unroll
                    for (int sb = 0; sb < SUB; ++sb)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {  // register e: rows g (e even), g + 8; keys 2 t, 2 t + 8
                            const float* x = &s[2 * sb + (e >> 1)][2 * (e & 1)];
                            const float mm = (e & 1) ? m1 : m0;
                            const float p0 = ptx::ex2(x[0] * p.scale_log2 - mm), p1 = ptx::ex2(x[1] * p.scale_log2 - mm);
                            l[e & 1] += p0 + p1;
                            constexpr float below = 1.f - 0x1p-23f;
                            const uint32_t hi = __byte_perm(__float_as_uint(p0 * below), __float_as_uint(p1 * below), 0x7632);
                            ph[sb][e] = hi;
                            pl[sb][e] = ptx::pack_bf16x2(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
                        }
                    // O += P V, two column pairs at a time: a product and its remainder's are four apart
#pragma unroll
                    for (int sb = 0; sb < SUB; ++sb)
#pragma unroll
                        for (int j = 0; j < D / 16; j += 2) {
                            uint32_t v0[4], v1[4];
                            ldsm4t((sv ^ (j * 32)) + sb * 16 * C::RB, v0);
                            ldsm4t((sv ^ ((j + 1) * 32)) + sb * 16 * C::RB, v1);
                            mma_16816(o[2 * j], ph[sb], v0[0], v0[1]);
                            mma_16816(o[2 * j + 1], ph[sb], v0[2], v0[3]);
                            mma_16816(o[2 * j + 2], ph[sb], v1[0], v1[1]);
                            mma_16816(o[2 * j + 3], ph[sb], v1[2], v1[3]);
                            mma_16816(o[2 * j], pl[sb], v0[0], v0[1]);
                            mma_16816(o[2 * j + 1], pl[sb], v0[2], v0[3]);
                            mma_16816(o[2 * j + 2], pl[sb], v1[0], v1[1]);
                            mma_16816(o[2 * j + 3], pl[sb], v1[2], v1[3]);
                        }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&empty[st]);
                if (++st == NST) st = 0, ++use;
            }

            // ---- join the warps: row statistics, then the scaled sums through the ring
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                if (t4 == 0) stat_m[slice * ROWS + rw * 16 + g8 + 8 * r] = m[r];
            }
            ptx::named_barrier_sync(1, NCONS);  // every stage is used, every maximum written
            float* join = reinterpret_cast<float*>(smem + C::OFF_RING);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = rw * 16 + g8 + 8 * r;
                float mt = stat_m[row];
#pragma unroll
                for (int k = 1; k < SLICES; ++k) mt = fmaxf(mt, stat_m[k * ROWS + row]);
                const float f = m[r] == -INFINITY ? 0.f : ptx::ex2(m[r] - mt);
                if (t4 == 0) stat_l[slice * ROWS + row] = l[r] * f;
                float* dst = join + (slice * ROWS + row) * C::RSTRIDE + 2 * t4;
#pragma unroll
                for (int x = 0; x < NT; ++x)
                    *reinterpret_cast<float2*>(dst + x * 8) = make_float2(o[x][2 * r] * f, o[x][2 * r + 1] * f);
            }
            ptx::named_barrier_sync(1, NCONS);
            const int c_first = whole ? 0 : walk.first_block();
            float* slot = whole ? nullptr : walk.slot(blockIdx.x, c_first);
            for (int x = tid; x < rows_here * (D / 4); x += NCONS) {
                const int row = x / (D / 4), q4 = x % (D / 4);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < SLICES; ++k) {
                    const float4 y = *reinterpret_cast<const float4*>(join + (k * ROWS + row) * C::RSTRIDE + q4 * 4);
                    acc.x += y.x, acc.y += y.y, acc.z += y.z, acc.w += y.w;
                }
                float lt = 0.f, mt = -INFINITY;
                if (whole || q4 == 0) {
#pragma unroll
                    for (int k = 0; k < SLICES; ++k) lt += stat_l[k * ROWS + row], mt = fmaxf(mt, stat_m[k * ROWS + row]);
                }
                if (whole) {
                    write_row4(p, row0 + row, D, q4, lt, acc);
                    if (q4 == 0 && p.lse != nullptr)
                        p.lse[row0 + row] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * 0.69314718055994531f;
                } else {
                    __stcg(reinterpret_cast<float4*>(slot + row * D) + q4, acc);
                    if (q4 == 0) {
                        __stcg(slot + p.rows_cap * D + row, mt);
                        __stcg(slot + p.rows_cap * D + p.rows_cap + row, lt);
                    }
                }
            }
            if (!whole) {
                // publish; the last block of the unit joins all of them
                ptx::named_barrier_sync(1, NCONS);
                const int c_last = walk.last_block();
                if (tid == 0) {
                    __threadfence();
                    const int ticket = atomicAdd(&p.tickets[c_first], 1);
                    const int last = ticket == c_last - c_first;
                    if (last) p.tickets[c_first] = 0;
                    *bcast = last;
                }
                ptx::named_barrier_sync(1, NCONS);
                if (*bcast) {
                    __threadfence();
                    const int parts = c_last - c_first + 1;
                    if (rows_here <= 2 * C::WARPS * (128 / D)) join_parts<D, C::WARPS, 1, 8>(p, walk.slot(c_first, c_first), walk.slot(c_first + 1, c_first), parts, row0, rows_here, warp, lane);
                    else join_parts<D, C::WARPS, 4, 2>(p, walk.slot(c_first, c_first), walk.slot(c_first + 1, c_first), parts, row0, rows_here, warp, lane);
                }
            }
        }
        it += n;
        ++n_units;
        ptx::fence_proxy_async_smem();  // the join's accesses to the ring come before the next loads
        __syncthreads();                // the join has been read, no wait is pending
        if (*abort_flag) return;
    }
}

}  // namespace e2d2
