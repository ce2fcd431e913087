// block_norm.hpp -- the block boundary, forward.
//
//     h  = y_0 + ... + y_{N-1}
//     p  = h r1 (w1 + o),   r1 = 1/sqrt(mean(h^2) + eps)
//     x' = beta x + alpha g p
//     z  = x' r2 (w2 + o),  r2 = 1/sqrt(mean(x'^2) + eps)
//
// Bound by memory: (N + 1) rows in, up to three out, and the weights, which
// stay in the caches.  One workgroup holds one row in registers from the
// loads to the stores, so that every byte moves once; both sums of squares
// are over values already there.  Only x' depends on r1, and its own sum is
// taken from the finished x' (from the sums of h^2, h x and x^2 it would lose
// all digits where the branch cancels the residual), so a row needs two
// workgroup sums.
#pragma once

#include "block_device.hpp"

namespace ptored {
namespace block {

template <int DT, int S, bool TAIL>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    __shared__ float red[2][1][kMaxWaves];
    const int stride = (int)blockDim.x * V;
    const int col0 = (int)threadIdx.x * V;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float h[S][V], x[S][V];
#pragma unroll
        for (int s = 0; s < S; ++s) {
#pragma unroll
            for (int i = 0; i < V; ++i) h[s][i] = 0.0f;
            load_slot<DT, TAIL>(a.x.p + row * a.x.ld, col0 + s * stride, a.cols, x[s]);
        }
        const int64_t part_off = row * a.part_ld;
#pragma unroll 4
        for (int r = 0; r < a.nranks; ++r) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float y[V];
                load_slot<DT, TAIL>(a.part[r] + part_off, col0 + s * stride, a.cols, y);
#pragma unroll
                for (int i = 0; i < V; ++i) h[s][i] += y[i];
            }
        }
        if (a.h.p != nullptr || a.kh.q != nullptr) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int col = col0 + s * stride;
                if (a.h.p) store_slot<DT, TAIL>(a.h.p + row * a.h.ld, col, a.cols, h[s]);
                if (a.kh.q) {
                    float t[V];
                    E::widen(E::narrow(h[s]), t);
                    pack_slot<V, TAIL>(a.kh, row, col, a.cols, t);
                }
            }
        }
        float branch = a.alpha;
        if (a.w1 != nullptr) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) sum[0] += h[s][i] * h[s][i];
            block_sum<1>(red[0], sum);
            const float r1 = 1.0f / sqrtf(sum[0] * a.inv_cols + a.eps);
            if (a.r1 != nullptr && threadIdx.x == 0) a.r1[row] = r1;
            branch *= r1;
        }
        const char* gate = nullptr;
        if (a.gate.p != nullptr) gate = a.gate.p + row / a.rows_per_gate * a.gate.ld;
        float sum[1] = {0.0f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int col = col0 + s * stride;
            float t[V];
#pragma unroll
            for (int i = 0; i < V; ++i) t[i] = branch * h[s][i];
            if (a.w1 != nullptr) {
                float w[V];
                load_weight<DT, TAIL>(a.w1, a.w_f32, a.offset, col, a.cols, w);
#pragma unroll
                for (int i = 0; i < V; ++i) t[i] *= w[i];
            }
            if (gate != nullptr) {
                float g[V];
                load_slot<DT, TAIL>(gate, col, a.cols, g);
#pragma unroll
                for (int i = 0; i < V; ++i) t[i] *= g[i];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[s][i] = a.beta * x[s][i] + t[i];
                sum[0] += x[s][i] * x[s][i];
            }
            if (a.x_out.p) store_slot<DT, TAIL>(a.x_out.p + row * a.x_out.ld, col, a.cols, x[s]);
            if (a.kx.q) {
                E::widen(E::narrow(x[s]), t);
                pack_slot<V, TAIL>(a.kx, row, col, a.cols, t);
            }
        }
        if (a.w2 == nullptr) continue;  // the same for every wave
        block_sum<1>(red[1], sum);
        const float r2 = 1.0f / sqrtf(sum[0] * a.inv_cols + a.eps);
        if (a.r2 != nullptr && threadIdx.x == 0) a.r2[row] = r2;
        if (a.z.p == nullptr && a.kz.q == nullptr) continue;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int col = col0 + s * stride;
            float w[V];
            load_weight<DT, TAIL>(a.w2, a.w_f32, a.offset, col, a.cols, w);
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] *= r2 * x[s][i];
            if (a.z.p) store_slot<DT, TAIL>(a.z.p + row * a.z.ld, col, a.cols, w);
            if (a.kz.q) {
                float t[V];
                E::widen(E::narrow(w), t);
                pack_slot<V, TAIL>(a.kz, row, col, a.cols, t);
            }
        }
    }
}

template <int DT, int S>
static int launch_norm(const NormArgs& a, int threads, hipStream_t stream) {
    const bool tail = a.cols % Elem<DT>::V != 0;
    const void* k = tail ? reinterpret_cast<const void*>(norm_kernel<DT, S, true>)
                         : reinterpret_cast<const void*>(norm_kernel<DT, S, false>);
    const int64_t grid = a.rows < (int64_t(1) << 30) ? a.rows : (int64_t(1) << 30);
    void* args[] = {const_cast<NormArgs*>(&a)};
    return hipLaunchKernel(k, dim3((uint32_t)grid), dim3((uint32_t)threads), args, 0, stream) ==
                   hipSuccess
               ? kOk
               : kFailed;
}

// The fewest slots per thread that 1024 threads reach, and no more threads
// than the row has slots.
template <int DT>
int norm_launch(const NormArgs& a, hipStream_t stream) {
    const int slots = (a.cols + Elem<DT>::V - 1) / Elem<DT>::V;
    int per = 1;
    while (slots > per * 1024) per *= 2;
    const int threads = ((slots + per - 1) / per + 63) / 64 * 64;
    if (per == 1) return launch_norm<DT, 1>(a, threads, stream);
    if (per == 2) return launch_norm<DT, 2>(a, threads, stream);
    if constexpr (Elem<DT>::V == 4) {
        if (per == 4) return launch_norm<DT, 4>(a, threads, stream);
    }
    return kFailed;  // more than PTORED_BLOCK_MAX_COLS columns
}

}  // namespace block
}  // namespace ptored
