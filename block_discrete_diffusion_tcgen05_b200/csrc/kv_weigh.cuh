// kv_weigh.cuh -- accumulated attention weight of a cache's rows: with the lse of an attention call,
//
//   weight_out_j = weight_j + sum_i exp(scale q_i . k_j - lse_i)      (i over the G S rows that read kv head h)
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "kv_paged.cuh"

namespace e2d2 {

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
