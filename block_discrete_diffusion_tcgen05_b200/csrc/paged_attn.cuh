// paged_attn.cuh -- the sampling step over a paged KV cache, and the accumulated attention weight of the
// cache's rows.
//
//   x_ij = scale q_i . k_j,  lse_i = log sum_j exp(x_ij),  out_i = sum_j exp(x_ij - lse_i) v_j
//
// for the S query rows of a block (one row: a single new token) and every query head, over the P[b] cached
// rows of the entry and, when given, the block's own S rows; and, with the lse of such a call,
//
//   weight_out_j = weight_j + sum_i exp(x_ij - lse_i)      (i over the G S rows that read kv head h)
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "kv_paged.cuh"

namespace e2d2 {

struct PagedAttnParams {
    PageView pages;
    const __nv_bfloat16* q;      // [B][Hq][S][D]
    const __nv_bfloat16* k;      // pools
    const __nv_bfloat16* v;
    const __nv_bfloat16* k_blk;  // [B][Hkv][S][D] or null
    const __nv_bfloat16* v_blk;
    const int* P_dev;
    __nv_bfloat16* out;          // [B][Hq][S][D]
    float* lse;                  // [B][Hq][S] or null
    int batch, q_heads, group, S;
    float scale_log2;            // softmax scale * log2(e)
};

// One block of four warps per query row: a warp takes every fourth key, a lane D/32 head dims; running
// maximum and sum per warp, joined at the end.
template <int D>
__global__ void __launch_bounds__(128) paged_attn_kernel(const __grid_constant__ PagedAttnParams p) {
    constexpr int E = D / 32;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const long long row = blockIdx.x;  // (b * Hq + hq) * S + s
    const int b = static_cast<int>(row / (static_cast<long long>(p.q_heads) * p.S));
    const int hq = static_cast<int>(row / p.S % p.q_heads);
    const int h = hq / p.group, Hkv = p.pages.kv_heads;
    const int P = ragged_clamp(__ldg(p.P_dev + b), p.pages.capacity());
    const int total = P + (p.k_blk != nullptr ? p.S : 0);
    float q[E], acc[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) {
        q[e] = __bfloat162float(p.q[row * D + lane * E + e]);
        acc[e] = 0.f;
    }
    for (int j = warp; j < total; j += 4) {
        const __nv_bfloat16 *kr, *vr;
        if (j < P) {
            const long long r = p.pages.pool_row(b, h, j);
            if (r < 0) continue;
            kr = p.k + r * D;
            vr = p.v + r * D;
        } else {
            const long long r = (static_cast<long long>(b) * Hkv + h) * p.S + (j - P);
            kr = p.k_blk + r * D;
            vr = p.v_blk + r * D;
        }
        float x = 0.f;
        for (int e = 0; e < E; ++e) x += q[e] * __bfloat162float(kr[lane * E + e]);
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        x *= p.scale_log2;
        const float mn = fmaxf(m, x);
        const float f = m == -INFINITY ? 0.f : ptx::ex2(m - mn), w = mn == -INFINITY ? 0.f : ptx::ex2(x - mn);
        l = l * f + w;
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + w * __bfloat162float(vr[lane * E + e]);
        m = mn;
    }
    __shared__ float sm[4], sl[4], so[4][D];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    __syncthreads();
    const float mt = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float lt = 0.f, f[4];
    for (int w = 0; w < 4; ++w) {
        f[w] = sm[w] == -INFINITY ? 0.f : ptx::ex2(sm[w] - mt);
        lt += sl[w] * f[w];
    }
    if (threadIdx.x < D) {
        float o = 0.f;
        for (int w = 0; w < 4; ++w) o += so[w][threadIdx.x] * f[w];
        p.out[row * D + threadIdx.x] = __float2bfloat16_rn(lt > 0.f ? o / lt : 0.f);
    }
    if (threadIdx.x == 0 && p.lse != nullptr)
        p.lse[row] = lt > 0.f ? (mt + log2f(lt)) * 0.69314718055994531f : -INFINITY;
}

struct WeighParams {
    PageView pages;
    const __nv_bfloat16* q;  // [B][Hq][S][D]
    const __nv_bfloat16* k;
    const int* P_dev;
    const float* lse;        // [B][Hq][S]
    const float* weight;     // [B][Hkv][capacity]
    float* weight_out;
    int batch, q_heads, group, S;
    float scale_log2;
};

// A warp per cached row (grid-stride over the rows of one (entry, kv head), blockIdx.y).
template <int D>
__global__ void __launch_bounds__(256) kv_weigh_kernel(const __grid_constant__ WeighParams p) {
    constexpr int E = D / 32;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int lane = threadIdx.x % 32;
    const int unit = blockIdx.y, Hkv = p.pages.kv_heads, cap = p.pages.capacity();
    const int b = unit / Hkv, h = unit % Hkv;
    const int P = ragged_clamp(__ldg(p.P_dev + b), cap);
    const int rows = p.group * p.S;
    const long long row0 = (static_cast<long long>(b) * p.q_heads + h * p.group) * p.S;
    for (int j = blockIdx.x * 8 + threadIdx.x / 32; j < P; j += gridDim.x * 8) {
        const long long r = p.pages.pool_row(b, h, j);
        float add = 0.f;
        if (r >= 0) {
            float k[E];
            for (int e = 0; e < E; ++e) k[e] = __bfloat162float(p.k[r * D + lane * E + e]);
            for (int i = 0; i < rows; ++i) {
                float x = 0.f;
                for (int e = 0; e < E; ++e) x += k[e] * __bfloat162float(p.q[(row0 + i) * D + lane * E + e]);
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                const float lse = p.lse[row0 + i];
                add += lse == -INFINITY ? 0.f : ptx::ex2(x * p.scale_log2 - lse * 1.4426950408889634f);
            }
        }
        if (lane == 0) {
            const long long w = static_cast<long long>(unit) * cap + j;
            p.weight_out[w] = p.weight[w] + add;
        }
    }
}

}  // namespace e2d2
