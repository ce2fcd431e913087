// block_norm_backward.hpp -- gradients of the block boundary.
//
//     xh = x' r2,  u = dz (w2 + o),  s = dx_out + r2 (u - xh mean(u xh))
//     dx = beta s,  dw2 = sum_t dz xh
//     hh = h r1,  e = alpha g s,  v = e (w1 + o)
//     dh = r1 (v - hh mean(v hh)),  dw1 = sum_t e hh,  dg = sum_t alpha p s
//
// With k = alpha g (w1 + o) hh, v hh = k s, so
//     mean(v hh) = mean(k (dx_out + r2 u)) - r2 mean(u xh) mean(k xh)
// and one workgroup sum of three values serves both norms: a row is read
// once, waits once, and is written.  The difference loses no more than s
// itself does, whose terms are the same.
//
// Bound by memory: four rows in (two of them may be packed), two out.  The
// column sums stay in registers while a workgroup walks a chunk of rows; each
// chunk leaves one partial row per sum in the workspace, and a second kernel
// adds those in a fixed order.
#pragma once

#include "block_device.hpp"

namespace ptored {
namespace block {

template <int DT, int S, bool TAIL, bool PACKED>
__global__ __launch_bounds__(1024) void grad_kernel(const GradArgs a) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    __shared__ float red[2][3][kMaxWaves];
    const int stride = (int)blockDim.x * V;
    const int col0 = (int)threadIdx.x * V;
    const int64_t chunk = blockIdx.x;
    const int64_t unit = chunk / a.chunks_per_unit;
    const int64_t begin = unit * a.unit_rows + (chunk - unit * a.chunks_per_unit) * a.chunk_rows;
    const int64_t unit_end = (unit + 1) * a.unit_rows;
    const int64_t end = begin + a.chunk_rows < unit_end ? begin + a.chunk_rows : unit_end;
    float aw1[S][V], aw2[S][V], ag[S][V];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) aw1[s][i] = aw2[s][i] = ag[s][i] = 0.0f;

    int turn = 0;
    for (int64_t row = begin; row < end; ++row, turn ^= 1) {
        const int64_t gate_row = a.gate.p != nullptr ? row / a.rows_per_gate : 0;
        const float r2 = a.w2 != nullptr ? a.r2[row] : 0.0f;
        const float r1 = a.w1 != nullptr ? a.r1[row] : 1.0f;
        float u[S][V], dxo[S][V], xh[S][V], hh[S][V], kw[S][V];
        float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int col = col0 + s * stride;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                u[s][i] = dxo[s][i] = xh[s][i] = hh[s][i] = 0.0f;
                kw[s][i] = a.alpha;
            }
            if (a.dxo.p) load_slot<DT, TAIL>(a.dxo.p + row * a.dxo.ld, col, a.cols, dxo[s]);
            if (a.w2) {
                load_slot<DT, TAIL>(a.dz.p + row * a.dz.ld, col, a.cols, u[s]);
                if constexpr (PACKED)
                    unpack_slot<V, TAIL>(a.kx, row, col, a.cols, xh[s]);
                else
                    load_slot<DT, TAIL>(a.x.p + row * a.x.ld, col, a.cols, xh[s]);
            }
            if (PACKED ? a.kh.q != nullptr : a.h.p != nullptr) {
                if constexpr (PACKED)
                    unpack_slot<V, TAIL>(a.kh, row, col, a.cols, hh[s]);
                else
                    load_slot<DT, TAIL>(a.h.p + row * a.h.ld, col, a.cols, hh[s]);
            }
            if (a.gate.p) {
                float g[V];
                load_slot<DT, TAIL>(a.gate.p + gate_row * a.gate.ld, col, a.cols, g);
#pragma unroll
                for (int i = 0; i < V; ++i) kw[s][i] *= g[i];
            }
            if (a.w2) {
                float w[V];
                load_weight<DT, TAIL>(a.w2, a.w_f32, a.offset, col, a.cols, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xh[s][i] *= r2;
                    aw2[s][i] += u[s][i] * xh[s][i];
                    u[s][i] *= w[i];
                    sum[0] += u[s][i] * xh[s][i];
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) hh[s][i] *= r1;
            if (a.w1) {
                float w[V];
                load_weight<DT, TAIL>(a.w1, a.w_f32, a.offset, col, a.cols, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float k = kw[s][i] * w[i] * hh[s][i];
                    sum[1] += k * (dxo[s][i] + r2 * u[s][i]);
                    sum[2] += k * xh[s][i];
                }
            }
        }
        if (a.w1 != nullptr || a.w2 != nullptr) block_sum<3>(red[turn], sum);
        const float c2 = sum[0] * a.inv_cols;
        const float c1 = (sum[1] - r2 * c2 * sum[2]) * a.inv_cols;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int col = col0 + s * stride;
            float d[V], dh[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                d[i] = dxo[s][i] + r2 * (u[s][i] - xh[s][i] * c2);  // s
                dh[i] = kw[s][i] * d[i];                            // e
            }
            if (a.w1) {
                float w[V];
                load_weight<DT, TAIL>(a.w1, a.w_f32, a.offset, col, a.cols, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    aw1[s][i] += dh[i] * hh[s][i];
                    ag[s][i] += a.alpha * d[i] * hh[s][i] * w[i];
                    dh[i] = r1 * (dh[i] * w[i] - hh[s][i] * c1);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) ag[s][i] += a.alpha * d[i] * hh[s][i];
            }
            if (a.dh.p) store_slot<DT, TAIL>(a.dh.p + row * a.dh.ld, col, a.cols, dh);
#pragma unroll
            for (int i = 0; i < V; ++i) d[i] *= a.beta;
            if (a.dx.p) store_slot<DT, TAIL>(a.dx.p + row * a.dx.ld, col, a.cols, d);
        }
        if (a.gate_direct && (row + 1) == (gate_row + 1) * a.rows_per_gate) {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                store_slot<DT, TAIL>(a.dgate.p + gate_row * a.dgate.ld, col0 + s * stride, a.cols,
                                     ag[s]);
#pragma unroll
                for (int i = 0; i < V; ++i) ag[s][i] = 0.0f;
            }
        }
    }
    // partial rows, 32 bits each
    const int64_t pitch = (int64_t)a.cols * 4;
    char* ws = reinterpret_cast<char*>(a.ws) + chunk * a.ws_slots * pitch;
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const int col = col0 + s * stride + i;
            if (a.slot_w1 >= 0)
                store_slot<PTORED_F32, TAIL>(ws + a.slot_w1 * pitch, col, a.cols, aw1[s] + i);
            if (a.slot_w2 >= 0)
                store_slot<PTORED_F32, TAIL>(ws + a.slot_w2 * pitch, col, a.cols, aw2[s] + i);
            if (a.slot_gate >= 0)
                store_slot<PTORED_F32, TAIL>(ws + a.slot_gate * pitch, col, a.cols, ag[s] + i);
        }
    }
}

// Adds partial rows: output row o (blockIdx.y: first dw1 and dw2 as wanted,
// then the gate rows) is the sum over its chunks.  64 columns a workgroup, 16
// partial sums of every 16th chunk each, joined in the LDS in a fixed order.
constexpr int kJoinCols = 64, kJoinParts = 16;

template <int DT>
__global__ __launch_bounds__(kJoinCols* kJoinParts) void grad_join_kernel(const GradArgs a,
                                                                         int64_t outputs) {
    __shared__ float part[kJoinParts][kJoinCols];
    const int lane = (int)threadIdx.x % kJoinCols, p = (int)threadIdx.x / kJoinCols;
    const int col = (int)blockIdx.x * kJoinCols + lane;
    const int weights = (a.slot_w1 >= 0) + (a.slot_w2 >= 0);
    for (int64_t o = blockIdx.y; o < outputs; o += gridDim.y) {
        int slot;
        int64_t first = 0, count = a.chunks;
        char* out;
        bool f32 = true;
        if (o < weights) {
            const bool is_w1 = a.slot_w1 >= 0 && o == 0;
            slot = is_w1 ? a.slot_w1 : a.slot_w2;
            out = is_w1 ? a.dw1 : a.dw2;
            f32 = a.w_f32 != 0;
        } else {
            slot = a.slot_gate;
            count = a.chunks_per_unit;
            first = (o - weights) * count;
            out = a.dgate.p + (o - weights) * a.dgate.ld;
            f32 = DT == PTORED_F32;
        }
        float sum = 0.0f;
        if (col < a.cols) {
            const float* ws = a.ws + (first * a.ws_slots + slot) * a.cols + col;
            const int64_t step = (int64_t)a.ws_slots * a.cols;
#pragma unroll 4
            for (int64_t c = p; c < count; c += kJoinParts) sum += ws[c * step];
        }
        part[p][lane] = sum;
        __syncthreads();
        if (p == 0 && col < a.cols) {
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < kJoinParts; ++i) total += part[i][lane];
            if (f32)
                Elem<PTORED_F32>::store1(out + (int64_t)col * 4, total);
            else
                Elem<DT>::store1(out + (int64_t)col * Elem<DT>::kBytes, total);
        }
        __syncthreads();
    }
}

template <int DT, int S, bool PACKED>
static int launch_grad(const GradArgs& a, int threads, hipStream_t stream) {
    const bool tail = a.cols % Elem<DT>::V != 0;
    const void* k = tail ? reinterpret_cast<const void*>(grad_kernel<DT, S, true, PACKED>)
                         : reinterpret_cast<const void*>(grad_kernel<DT, S, false, PACKED>);
    void* args[] = {const_cast<GradArgs*>(&a)};
    return hipLaunchKernel(k, dim3((uint32_t)a.chunks), dim3((uint32_t)threads), args, 0,
                           stream) == hipSuccess
               ? kOk
               : kFailed;
}

template <int DT>
int grad_launch(const GradArgs& a, hipStream_t stream) {
    const int slots = (a.cols + Elem<DT>::V - 1) / Elem<DT>::V;
    int per = 1;
    while (slots > per * 1024) per *= 2;
    const int threads = ((slots + per - 1) / per + 63) / 64 * 64;
    const bool packed = a.kx.q != nullptr || a.kh.q != nullptr;
    int rc = a.chunks > 0 ? kFailed : kOk;
    if (a.chunks > 0) {
        if (per == 1)
            rc = packed ? launch_grad<DT, 1, true>(a, threads, stream)
                        : launch_grad<DT, 1, false>(a, threads, stream);
        else if (per == 2)
            rc = packed ? launch_grad<DT, 2, true>(a, threads, stream)
                        : launch_grad<DT, 2, false>(a, threads, stream);
        if constexpr (Elem<DT>::V == 4) {
            if (per == 4)
                rc = packed ? launch_grad<DT, 4, true>(a, threads, stream)
                            : launch_grad<DT, 4, false>(a, threads, stream);
        }
    }
    if (rc != kOk) return rc;
    int64_t outputs = (a.slot_w1 >= 0) + (a.slot_w2 >= 0);
    if (a.slot_gate >= 0) outputs += a.gate_rows;
    if (outputs == 0) return kOk;
    const dim3 grid((uint32_t)((a.cols + kJoinCols - 1) / kJoinCols),
                    (uint32_t)(outputs < 32768 ? outputs : 32768));
    void* args[] = {const_cast<GradArgs*>(&a), &outputs};
    return hipLaunchKernel(reinterpret_cast<const void*>(grad_join_kernel<DT>), grid,
                           dim3(kJoinCols * kJoinParts), args, 0, stream) == hipSuccess
               ? kOk
               : kFailed;
}

}  // namespace block
}  // namespace ptored
