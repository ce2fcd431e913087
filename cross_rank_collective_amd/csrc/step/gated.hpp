// gated.hpp -- the activations of the gated feed-forward block, and the
// gradients that its products start from.
//
//     dg = dy u f'(g),  du = dy f(g)
//
// Bound by memory: three matrices in, two out (8192 x 8192 bf16 115-122 us, 5.5-5.8
// TB/s).  dg and du are outputs that the products read, rounded to the type: what
// a training step keeps of them, and what its products in that type would read.
#pragma once

#include <algorithm>

#include "block/block_device.hpp"
#include "step_plan.h"

namespace ptored {
namespace step {

using namespace block;

// f(g) = g s(g) for all three: s is the logistic function, the normal
// distribution's, or the logistic function of 2 sqrt(2/pi) (g + 0.044715 g^3),
// since (1 + tanh(t)) / 2 is that of 2t.
//
// For 16-bit types the logistic function is the hardware's 2^v and reciprocal:
// off by some (4 + 2 |v|) 2^-24 (v's product with log2(e) is rounded), at most
// 2^-16, where the type rounds by 2^-8 or 2^-11, and 3% off the whole forward pass
// of 2048 tokens (235 -> 226 us).  In either form it is 0 where it would be below
// 2^-128, and may be below 2^-126.
template <int DT>
__device__ __forceinline__ float logistic(float v) {
    if constexpr (DT == PTORED_F32)
        return 1.0f / (1.0f + expf(-v));
    else
        return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504f));
}
__device__ __forceinline__ float normal_cdf(float g) { return 0.5f * erfcf(g * -0.70710678f); }
constexpr float kTanhScale = 1.59576912f;  // 2 sqrt(2/pi)
template <int DT>
__device__ __forceinline__ float activation(int which, float g) {
    switch (which) {
        case PTORED_SILU: return g * logistic<DT>(g);
        case PTORED_GELU: return g * normal_cdf(g);
        default: return g * logistic<DT>(kTanhScale * (g + 0.044715f * g * g * g));
    }
}
// f(g) and f'(g).
template <int DT>
__device__ __forceinline__ void with_slope(int which, float g, float& f, float& slope) {
    switch (which) {
        case PTORED_SILU: {
            const float s = logistic<DT>(g);
            f = g * s;
            slope = s * (1.0f + g * (1.0f - s));
            break;
        }
        case PTORED_GELU: {
            const float s = normal_cdf(g);
            f = g * s;
            slope = s + g * (0.39894228f * expf(-0.5f * g * g));
            break;
        }
        default: {
            const float s = logistic<DT>(kTanhScale * (g + 0.044715f * g * g * g));
            const float q = s * (1.0f - s);
            f = g * s;
            // where the logistic function is flat, g^2 may be infinite
            slope = q == 0.0f ? s : s + g * q * (kTanhScale * (1.0f + 0.134145f * g * g));
        }
    }
}

constexpr int kSlopeThreads = 256;

template <int DT, int EDGE>
__global__ __launch_bounds__(kSlopeThreads) void slope_kernel(const SlopeArgs a) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    const int64_t slots = (a.cols + V - 1) / V;
    const int64_t items = a.rows * slots;
    for (int64_t i = (int64_t)blockIdx.x * kSlopeThreads + threadIdx.x; i < items;
         i += (int64_t)gridDim.x * kSlopeThreads) {
        const int64_t row = i / slots, col = (i - row * slots) * V;
        const int64_t at = col * E::kBytes;
        const int n = EDGE == kWhole || col + V <= a.cols ? V : (int)(a.cols - col);
        auto load = [&](const Mat& m, float* v) {
            const char* p = m.p + row * m.ld + at;
            if (EDGE == kWhole || n == V) {
                E::widen(*reinterpret_cast<const u32x4_any*>(p), v);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) v[k] = k < n ? E::load1(p + k * E::kBytes) : 0.0f;
            }
        };
        auto store = [&](const Mat& m, const float* v) {
            char* p = m.p + row * m.ld + at;
            if (EDGE == kWhole || n == V) {
                *reinterpret_cast<u32x4_any*>(p) = E::narrow(v);
            } else {
#pragma unroll
                for (int k = 0; k < V - 1; ++k)
                    if (k < n) E::store1(p + k * E::kBytes, v[k]);
            }
        };
        float dy[V], g[V], u[V];
        load(a.dy, dy);
        load(a.gate, g);
        load(a.up, u);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float f, slope;
            with_slope<DT>(a.activation, g[k], f, slope);
            g[k] = dy[k] * u[k] * slope;
            u[k] = dy[k] * f;
        }
        store(a.dgate, g);
        store(a.dup, u);
    }
}

template <int DT>
int slope_launch(const SlopeArgs& a, hipStream_t stream) {
    constexpr int V = Elem<DT>::V;
    const void* k = a.cols % V == 0 ? reinterpret_cast<const void*>(slope_kernel<DT, kWhole>)
                                    : reinterpret_cast<const void*>(slope_kernel<DT, kPart>);
    const int64_t items = a.rows * ((a.cols + V - 1) / V);
    const int64_t grid = std::min<int64_t>((items + kSlopeThreads - 1) / kSlopeThreads, 1 << 20);
    void* args[] = {const_cast<SlopeArgs*>(&a)};
    return hipLaunchKernel(k, dim3((uint32_t)grid), dim3(kSlopeThreads), args, 0, stream) == hipSuccess
               ? kOk
               : kFailed;
}

}  // namespace step
}  // namespace ptored
