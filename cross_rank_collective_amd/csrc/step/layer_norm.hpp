// layer_norm.hpp -- the boundary of a block with layer norm, and its gradients.
//
//     x' = x + y_0 + ... + y_{N-1}
//     m  = mean(x'),  r = 1/sqrt(mean((x' - m)^2) + eps),  z = (x' - m) r w + b
//
//     xh = (x' - m) r,  u = dz w
//     dx = dx_out + r (u - mean(u) - xh mean(u xh)),  dw = sum_t dz xh,  db = sum_t dz
//
// Bound by memory.  Forward: a workgroup holds a row in registers from the
// loads to the stores.  The variance is the mean of squares of differences
// from the mean, not mean(x'^2) - m^2, which would lose all digits of a row
// whose mean is far from zero; so a row needs two workgroup sums.  The first
// sum's rounding leaves the differences a common error c; their own sum, taken
// along with the squares', gives c, which is then put right in m, r and z.
//
// Gradients: a workgroup walks every chunks-th row, the next row's loads in
// flight while the current one waits for its sum, and keeps the column sums of
// dw and db in registers.  Each leaves one partial row of either in the
// workspace; a second kernel adds those in a fixed order.
//
// Measured (bf16, one pass among others): forward, 8192 x 4096, 4 partials, 80 us,
// 5.9 TB/s, where a large copy reaches 6.2; 1 x 8192, 8 partials, 5.2 us, a launch
// and one chain of loads, two sums and stores.  Gradients, 16384 x 4096: 97 us and
// 4.8 for the sums over the chunks, 5.3 TB/s; 1777 x 1003 f16 12.5 us, two launches.
#pragma once

#include <algorithm>

#include "block/block_device.hpp"
#include "step_plan.h"

namespace ptored {
namespace step {

using namespace block;

// An infinity or a NaN: what a sum is whose parts passed binary32's range, a NaN
// where they passed it both ways.
__device__ __forceinline__ bool past_range(float v) { return (as_u(v) & 0x7F800000u) == 0x7F800000u; }
constexpr float kMost = 0x1.fffffep127f;  // binary32's

// S slots of a row per thread.
template <int DT, int S, int EDGE>
__global__ __launch_bounds__(1024) void layer_norm_kernel(const LayerNormArgs a) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    constexpr int R = 4;  // ranks whose slots are in flight together
    typedef Slots<DT, S, EDGE> Row;
    __shared__ f32x4 red[2][2][kMaxWaves / 4];
    const Row t(a.cols);
    // elements of the last slot that are inside the row
    const int inside = a.cols - t.col(S - 1);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        float v[S][V];
        {
            const rsrc_t x_row = t.row(a.x.p + row * a.x.ld);
            u32x4 raw[S];
#pragma unroll
            for (int s = 0; s < S; ++s) raw[s] = t.load(x_row, s);
#pragma unroll
            for (int s = 0; s < S; ++s) t.take(raw[s], s, v[s]);
        }
        const int64_t part_off = row * a.part_ld;
        for (int r0 = 0; r0 < a.nranks; r0 += R) {
            u32x4 y_raw[R][S];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                // past the last rank nothing is read and zeros are added
                const bool in = r0 + r < a.nranks;
                const rsrc_t y_row =
                    row_rsrc(a.part[in ? r0 + r : 0] + part_off, in ? a.cols * E::kBytes : 0);
#pragma unroll
                for (int s = 0; s < S; ++s) y_raw[r][s] = t.load(y_row, s);
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    float y[V];
                    t.take(y_raw[r][s], s, y);
#pragma unroll
                    for (int i = 0; i < V; ++i) v[s][i] += y[i];
                }
        }
        const auto& b = args_again<LayerNormArgs>();
        // asked for before the sums are waited for
        typename Row::Weight w[S], bias[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            w[s] = t.load_weight(b.w, b.w_f32, s);
            bias[s] = t.load_weight(b.b, b.w_f32, s);
        }
        if (b.x_out.p) {
            const rsrc_t out = t.row(b.x_out.p + row * b.x_out.ld);
#pragma unroll
            for (int s = 0; s < S; ++s) t.store(out, s, v[s]);
        }
        if (b.z.p == nullptr && b.mean == nullptr && b.rstd == nullptr) continue;
        // slots past the row hold zeros
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) sum[0] += v[s][i];
        block_sum<1>(red[turn], sum);
        turn ^= 1;
        float m = sum[0] * b.inv_cols;
        if (__builtin_expect(past_range(as_f((uint32_t)__builtin_amdgcn_readfirstlane((int)as_u(sum[0])))), 0)) {
            // the sum passes binary32's range where the mean may not
            sum[0] = 0.0f;
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) sum[0] += v[s][i] * b.inv_cols;
            block_sum<1>(red[turn], sum);
            turn ^= 1;
            m = sum[0];
        }
        sum[0] = sum[1] = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[s][i] = s < S - 1 || i < inside ? v[s][i] - m : 0.0f;
                sum[0] += v[s][i];
                sum[1] += v[s][i] * v[s][i];
            }
        block_sum<2>(red[turn], sum);
        turn ^= 1;
        float c = sum[0] * b.inv_cols, var = sum[1] * b.inv_cols;
        if (__builtin_expect(past_range(as_f((uint32_t)__builtin_amdgcn_readfirstlane((int)as_u(sum[1])))), 0)) {
            sum[0] = sum[1] = 0.0f;
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float part = v[s][i] * b.inv_cols;
                    sum[0] += part;
                    sum[1] += part * v[s][i];
                }
            block_sum<2>(red[turn], sum);
            turn ^= 1;
            // Where a difference itself passes the range there is no c: m stands as it
            // is, and as the variance's r is 0, the range's end does for the difference.
            c = past_range(sum[0]) ? 0.0f : sum[0];
            var = sum[1];
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    v[s][i] = __builtin_fabsf(v[s][i]) > kMost ? __builtin_copysignf(kMost, v[s][i]) : v[s][i];
        }
        var -= c * c;
        var = var < 0.0f ? 0.0f : var;  // a NaN stays
        const float r = 1.0f / sqrtf(var + b.eps);
        const auto& d = args_again<LayerNormArgs>();
        if (threadIdx.x == 0) {
            if (d.mean != nullptr) d.mean[row] = m + c;
            if (d.rstd != nullptr) d.rstd[row] = r;
        }
        if (d.z.p == nullptr) continue;
        const rsrc_t z_row = t.row(d.z.p + row * d.z.ld);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float z[V], k[V];
            t.take_weight(w[s], d.w_f32, d.w != nullptr ? 0.0f : 1.0f, s, z);
            t.take_weight(bias[s], d.w_f32, 0.0f, s, k);
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = (v[s][i] - c) * r * z[i] + k[i];
            t.store(z_row, s, z);
        }
    }
}

template <int DT, int S>
static const void* layer_norm_pick(int cols) {
    switch (edge_of<DT>(cols)) {
        case kWhole: return reinterpret_cast<const void*>(layer_norm_kernel<DT, S, kWhole>);
        case kPart: return reinterpret_cast<const void*>(layer_norm_kernel<DT, S, kPart>);
        default: return reinterpret_cast<const void*>(layer_norm_kernel<DT, 1, kTiny>);
    }
}

inline int launched(hipError_t e) { return e == hipSuccess ? kOk : kFailed; }

template <int DT>
int layer_norm_launch(const LayerNormArgs& a, hipStream_t stream) {
    constexpr int V = Elem<DT>::V;
    const int slots = (a.cols + V - 1) / V;
    // 16 elements a thread, 8 where the rows leave compute units idle anyway
    int per = (a.rows <= 256 ? 8 : 16) / V;
    while (slots > per * 1024) per *= 2;
    const int threads = slot_threads(slots, per);
    const void* k = per == 1 ? layer_norm_pick<DT, 1>(a.cols) : layer_norm_pick<DT, 2>(a.cols);
    if constexpr (V == 4) {
        if (per == 4) k = layer_norm_pick<DT, 4>(a.cols);
    }
    // a launch takes fewer than 2^32 threads
    const int64_t grid = std::min<int64_t>(a.rows, (int64_t(1) << 31) / threads);
    void* args[] = {const_cast<LayerNormArgs*>(&a)};
    return launched(hipLaunchKernel(k, dim3((uint32_t)grid), dim3((uint32_t)threads), args, 0, stream));
}

// ---------------------------------------------------------------- gradients

template <int DT, int S, int EDGE>
__global__ __launch_bounds__(1024) void layer_grad_kernel(const LayerGradArgs a) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    // Up to 8 elements a thread (8192 columns) the weight is kept in registers
    // and the next row is loaded ahead; with more neither fits the 128 that
    // 1024 threads leave to one.
    constexpr bool HOLD = S * V <= 8;
    typedef Slots<DT, S, EDGE> Row;
    __shared__ f32x4 red[2][2][kMaxWaves / 4];
    const Row t(a.cols);
    const int row_bytes = a.cols * E::kBytes;

    struct Raw {
        u32x4 dz[S], dxo[S], x[S];
        float m, r;
    };
    auto load = [&](int64_t row, Raw& to) {
        const bool in = row < a.rows;
        const int64_t at = in ? row : 0;
        const int bytes = in ? row_bytes : 0;
        const rsrc_t z = row_rsrc(a.dz.p + at * a.dz.ld, bytes);
        const rsrc_t x = row_rsrc(a.x.p + at * a.x.ld, bytes);
        const rsrc_t d = row_rsrc(a.dxo.p + at * a.dxo.ld, a.dxo.p != nullptr ? bytes : 0);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            to.dz[s] = t.load(z, s);
            to.x[s] = t.load(x, s);
            to.dxo[s] = t.load(d, s);
        }
        to.m = a.mean[at];
        to.r = a.rstd[at];
    };
    const float one = a.w != nullptr ? 0.0f : 1.0f;
    typename Row::Weight w_raw[S];
#pragma unroll
    for (int s = 0; s < S; ++s) w_raw[s] = t.load_weight(a.w, a.w_f32, s);
    Raw raw, other;
    if constexpr (HOLD) load(blockIdx.x, raw);
    float w[S][V], sw[S][V], sb[S][V];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if constexpr (HOLD) t.take_weight(w_raw[s], a.w_f32, one, s, w[s]);
#pragma unroll
        for (int i = 0; i < V; ++i) sw[s][i] = sb[s][i] = 0.0f;
    }
    int turn = 0;
    auto one_row = [&](int64_t row, Raw& raw, Raw& next) {
        if constexpr (!HOLD) load(row, raw);
        const float r = raw.r;
        float u[S][V], xh[S][V], sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            t.take(raw.dz[s], s, u[s]);
            t.take(raw.x[s], s, xh[s]);
            float k[V];
            if constexpr (!HOLD)
                t.take_weight(t.load_weight(a.w, a.w_f32, s), a.w_f32, one, s, k);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // past the row dz is zero, and so is all that depends on it
                xh[s][i] = (xh[s][i] - raw.m) * r;
                sw[s][i] += u[s][i] * xh[s][i];
                sb[s][i] += u[s][i];
                u[s][i] *= HOLD ? w[s][i] : k[i];
                sum[0] += u[s][i];
                sum[1] += u[s][i] * xh[s][i];
            }
        }
        if constexpr (HOLD) load(row + a.chunks, next);
        if (a.dx.p == nullptr) return;
        block_sum<2>(red[turn], sum);
        turn ^= 1;
        const float c0 = sum[0] * a.inv_cols, c1 = sum[1] * a.inv_cols;
        const rsrc_t out = t.row(a.dx.p + row * a.dx.ld);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float d[V];
            t.take(raw.dxo[s], s, d);
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] += r * (u[s][i] - c0 - xh[s][i] * c1);
            t.store(out, s, d);
        }
    };
    // two rows a turn, each loading the other's: nothing is copied between them
    for (int64_t row = blockIdx.x; row < a.rows; row += 2 * a.chunks) {
        one_row(row, raw, other);
        if (row + a.chunks >= a.rows) break;
        one_row(row + a.chunks, other, raw);
    }
    const auto& z = args_again<LayerGradArgs>();
    if (z.ws == nullptr) return;
    float* ws = z.ws + (int64_t)blockIdx.x * 2 * z.ws_pitch;
    auto leave = [&](float* p, float (*v)[V]) {
        const rsrc_t to = row_rsrc(p, (int)z.ws_pitch * 4);
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < V; i += 4)
                __builtin_amdgcn_raw_buffer_store_b128(
                    (u32x4){as_u(v[s][i]), as_u(v[s][i + 1]), as_u(v[s][i + 2]), as_u(v[s][i + 3])},
                    to, (t.col(s) + i) * 4, 0, 0);
    };
    if (z.dw != nullptr) leave(ws, sw);
    if (z.db != nullptr) leave(ws + z.ws_pitch, sb);
}

// dw and db (blockIdx.y, as wanted): the chunks' partial rows added.  A
// workgroup takes COLS columns in lanes of 4 and 4096 / COLS partial sums, one
// for each chunk of a stride, joined in the LDS in a fixed order.
template <int DT, int COLS>
__global__ __launch_bounds__(1024) void layer_join_kernel(const LayerGradArgs a) {
    constexpr int kLanes = COLS / 4, kParts = 1024 / kLanes;
    __shared__ f32x4 part[kParts][kLanes];
    const int lane = (int)threadIdx.x % kLanes, p = (int)threadIdx.x / kLanes;
    const int col = (int)blockIdx.x * COLS + lane * 4;
    const bool is_w = a.dw != nullptr && blockIdx.y == 0;
    f32x4 sum = (f32x4)(0.0f);
    if (col < a.cols) {
        const float* ws = a.ws + (is_w ? 0 : a.ws_pitch) + col;
#pragma unroll 8
        for (int64_t c = p; c < a.chunks; c += kParts)
            sum += *reinterpret_cast<const f32x4*>(ws + c * 2 * a.ws_pitch);
    }
    part[p][lane] = sum;
    __syncthreads();
#pragma unroll
    for (int half = kParts / 2; half >= 1; half /= 2) {
        if (p < half) part[p][lane] += part[p + half][lane];
        __syncthreads();
    }
    const int c = (int)threadIdx.x, at = (int)blockIdx.x * COLS + c;
    if (c < COLS && at < a.cols) {
        const float total = part[0][c / 4][c % 4];
        char* out = is_w ? a.dw : a.db;
        if (a.w_f32)
            Elem<PTORED_F32>::store1(out + (int64_t)at * 4, total);
        else
            Elem<DT>::store1(out + (int64_t)at * Elem<DT>::kBytes, total);
    }
}

template <int DT, int S>
static const void* layer_grad_pick(int cols) {
    switch (edge_of<DT>(cols)) {
        case kWhole: return reinterpret_cast<const void*>(layer_grad_kernel<DT, S, kWhole>);
        case kPart: return reinterpret_cast<const void*>(layer_grad_kernel<DT, S, kPart>);
        default: return reinterpret_cast<const void*>(layer_grad_kernel<DT, 1, kTiny>);
    }
}

template <int DT>
int layer_grad_launch(const LayerGradArgs& a, hipStream_t stream) {
    constexpr int V = Elem<DT>::V;
    void* args[] = {const_cast<LayerGradArgs*>(&a)};
    if (a.chunks > 0) {
        const int slots = (a.cols + V - 1) / V;
        int per = 1;
        while (slots > per * 1024) per *= 2;
        const int threads = slot_threads(slots, per);
        const void* k = per == 1 ? layer_grad_pick<DT, 1>(a.cols) : layer_grad_pick<DT, 2>(a.cols);
        if constexpr (V == 4) {
            if (per == 4) k = layer_grad_pick<DT, 4>(a.cols);
        }
        const int rc = launched(hipLaunchKernel(k, dim3((uint32_t)a.chunks), dim3((uint32_t)threads),
                                                args, 0, stream));
        if (rc != kOk) return rc;
    }
    const uint32_t outputs = (a.dw != nullptr) + (a.db != nullptr);
    if (outputs == 0) return kOk;
    // fewer columns a workgroup where there would be few workgroups
    const int64_t groups = a.chunks > 64 ? (int64_t)((a.cols + 63) / 64) * outputs : 256;
    const int cols = groups <= 32 ? 16 : groups <= 112 ? 32 : 64;
    const void* k = cols == 16   ? reinterpret_cast<const void*>(layer_join_kernel<DT, 16>)
                    : cols == 32 ? reinterpret_cast<const void*>(layer_join_kernel<DT, 32>)
                                 : reinterpret_cast<const void*>(layer_join_kernel<DT, 64>);
    return launched(hipLaunchKernel(k, dim3((uint32_t)((a.cols + cols - 1) / cols), outputs),
                                    dim3(1024), args, 0, stream));
}

}  // namespace step
}  // namespace ptored
