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
// Bound by memory: four rows in (two of them may be packed), two out.  A
// workgroup walks a chunk of rows, the next row's loads in flight while the
// current one waits for its sum.  The weights' and the gate's gradients share
// one column sum: with A = sum_t s hh over the rows of one gate row,
// dg = alpha (w1 + o) A and that gate row adds alpha g A to dw1.  Each chunk
// leaves one partial row per sum in the workspace, and a second kernel adds
// those in a fixed order.
#pragma once

#include "block_device.hpp"

namespace ptored {
namespace block {

// A packed or whole activation's slot as loaded.
template <bool PACKED>
struct Activation {
    u32x4 w;
};
template <>
struct Activation<true> {
    KeptRaw w;
};

// MANY: a chunk holds several gate rows; otherwise A alone tells their
// gradients at the chunk's end.
template <int DT, int S, int EDGE, bool PACKED, bool MANY>
__global__ __launch_bounds__(1024) void grad_kernel(const GradArgs a) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    // Up to 8 elements a thread, the factors that rows share stay in registers
    // and the next row is loaded ahead; with more neither fits.
    constexpr bool HOLD = S * V <= 8;
    typedef Slots<DT, S, EDGE> Row;
    __shared__ f32x4 red[2][3][kMaxWaves / 4];
    const Row t(a.cols);
    const int64_t chunk = blockIdx.x;
    const int64_t unit = chunk / a.chunks_per_unit;
    const int64_t begin = unit * a.unit_rows + (chunk - unit * a.chunks_per_unit) * a.chunk_rows;
    const int64_t unit_end = (unit + 1) * a.unit_rows;
    const int64_t end = begin + a.chunk_rows < unit_end ? begin + a.chunk_rows : unit_end;
    const bool pre = a.w2 != nullptr, post = a.w1 != nullptr, gated = a.gate.p != nullptr;
    const bool has_h = PACKED ? a.kh.q != nullptr : a.h.p != nullptr;

    // what a row is made of, as loaded; absent rows read as zeros
    struct Raw {
        u32x4 dz[S], dxo[S];
        Activation<PACKED> x[S], h[S];
        float r1, r2;
    };
    auto activation = [&](const Mat& m, const Kept& k, int64_t row, bool there,
                          Activation<PACKED>* to) {
        if constexpr (PACKED) {
            typename Row::KeptRow r = t.kept_row(k, there ? row : 0);
            if (!there) r.q = r.s = row_rsrc(nullptr, 0);
#pragma unroll
            for (int s = 0; s < S; ++s) to[s].w = t.load_kept(r, s);
        } else {
            const rsrc_t r = there ? t.row(m.p + row * m.ld) : row_rsrc(nullptr, 0);
#pragma unroll
            for (int s = 0; s < S; ++s) to[s].w = t.load(r, s);
        }
    };
    auto load = [&](int64_t row, Raw& to) {
        const rsrc_t dz = pre ? t.row(a.dz.p + row * a.dz.ld) : row_rsrc(nullptr, 0);
        const rsrc_t dxo = a.dxo.p ? t.row(a.dxo.p + row * a.dxo.ld) : row_rsrc(nullptr, 0);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            to.dz[s] = t.load(dz, s);
            to.dxo[s] = t.load(dxo, s);
        }
        activation(a.x, a.kx, row, pre, to.x);
        activation(a.h, a.kh, row, has_h, to.h);
        to.r2 = pre ? a.r2[row] : 0.0f;
        to.r1 = post ? a.r1[row] : 1.0f;
    };
    // an activation times its row's reciprocal norm
    auto take = [&](const Activation<PACKED>& w, int s, float by, float* v) {
        if constexpr (PACKED) {
            t.take_kept(w.w, s, by, v);
        } else {
            t.take(w.w, s, v);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= by;
        }
    };
    auto weight = [&](const char* w, int s, float* v) {
        if (w != nullptr) {
            t.take_weight(t.load_weight(w, a.w_f32, s), a.w_f32, a.offset, s, v);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = 1.0f;
        }
    };
    auto load_gate = [&](int64_t gate_row, u32x4* to) {
        const rsrc_t r = t.row(a.gate.p + gate_row * a.gate.ld);
#pragma unroll
        for (int s = 0; s < S; ++s) to[s] = t.load(r, s);
    };
    auto take_gate = [&](const u32x4* from, int s, float* v) {  // alpha g
        if (gated) {
            t.take(from[s], s, v);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= a.alpha;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = a.alpha;
        }
    };

    int64_t gate_row = gated ? begin / a.rows_per_gate : 0;
    int64_t gate_end = MANY ? (gate_row + 1) * a.rows_per_gate : end;
    u32x4 gate[S];  // MANY: of the next row, where that begins a gate row
    if (gated) load_gate(gate_row, gate);
    // HOLD: w2 + o; alpha g; alpha g (w1 + o), or with MANY w1 + o
    float w2[S][V], ag[S][V], kw[S][V];
    if constexpr (HOLD) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            weight(a.w2, s, w2[s]);
            weight(a.w1, s, kw[s]);
            if constexpr (!MANY) {
                take_gate(gate, s, ag[s]);
#pragma unroll
                for (int i = 0; i < V; ++i) kw[s][i] *= ag[s][i];
            }
        }
    }
    // alpha g (w1 + o) of the current row
    auto scale = [&](int s, float* v) {
        if constexpr (!HOLD) {
            float g[V];
            weight(a.w1, s, v);
            take_gate(gate, s, g);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= g[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = MANY ? ag[s][i] * kw[s][i] : kw[s][i];
        }
    };
    float sw1[S][V], sw2[S][V], sa[S][V];  // dw1 (MANY), dw2, A
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) sw1[s][i] = sw2[s][i] = sa[s][i] = 0.0f;

    int turn = 0;
    Raw next;
    if constexpr (HOLD) load(begin, next);
    bool fresh = MANY;  // the row begins a gate row, or the chunk
    for (int64_t row = begin; row < end; ++row, turn ^= 1) {
        if constexpr (!HOLD) {
            load(row, next);
            if (MANY && fresh) load_gate(gate_row, gate);
        }
        if (HOLD && MANY && fresh) {
#pragma unroll
            for (int s = 0; s < S; ++s) take_gate(gate, s, ag[s]);
        }
        const float r1 = next.r1, r2 = next.r2;
        float dxo[S][V], xh[S][V], hh[S][V];
        float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float u[V], k[V];
            t.take(next.dz[s], s, u);
            t.take(next.dxo[s], s, dxo[s]);
            take(next.x[s], s, r2, xh[s]);
            take(next.h[s], s, r1, hh[s]);
            scale(s, k);
            if constexpr (!HOLD) weight(a.w2, s, w2[s]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sw2[s][i] += u[i] * xh[s][i];
                u[i] *= w2[s][i];
                dxo[s][i] += r2 * u[i];
                sum[0] += u[i] * xh[s][i];
                k[i] *= hh[s][i];
                sum[1] += k[i] * dxo[s][i];
                sum[2] += k[i] * xh[s][i];
            }
        }
        fresh = MANY && row + 1 == gate_end;
        if (HOLD && row + 1 < end) {
            load(row + 1, next);
            if (fresh) load_gate(gate_row + 1, gate);
        }
        if (post || pre) block_sum<3>(red[turn], sum);
        const float c2 = r2 * sum[0] * a.inv_cols;
        const float c1 = r1 * ((sum[1] - c2 * sum[2]) * a.inv_cols);
        const rsrc_t dh_row = a.dh.p ? t.row(a.dh.p + row * a.dh.ld) : row_rsrc(nullptr, 0);
        const rsrc_t dx_row = a.dx.p ? t.row(a.dx.p + row * a.dx.ld) : row_rsrc(nullptr, 0);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float dh[V], k[V];
            scale(s, k);
            if constexpr (MANY && !HOLD) take_gate(gate, s, ag[s]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = dxo[s][i] - xh[s][i] * c2;  // s
                const float e = d * hh[s][i];
                sa[s][i] += e;
                if constexpr (MANY) sw1[s][i] += ag[s][i] * e;
                dh[i] = r1 * (k[i] * d);
                dxo[s][i] = a.beta * d;
            }
            if (post) {
#pragma unroll
                for (int i = 0; i < V; ++i) dh[i] -= hh[s][i] * c1;
            }
            if (a.dh.p) t.store(dh_row, s, dh);
            if (a.dx.p) t.store(dx_row, s, dxo[s]);
        }
        if (MANY && (fresh || row + 1 == end)) {
            if (a.gate_direct) {
                const rsrc_t r = t.row(a.dgate.p + gate_row * a.dgate.ld);
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    float w[V];
                    if constexpr (!HOLD) weight(a.w1, s, w);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        sa[s][i] *= a.alpha * (HOLD ? kw[s][i] : w[i]);
                    }
                    t.store(r, s, sa[s]);
                }
            }
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) sa[s][i] = 0.0f;
            gate_row += 1;
            gate_end += a.rows_per_gate;
        }
    }
    if constexpr (!MANY) {
        const rsrc_t dg =
            a.gate_direct ? t.row(a.dgate.p + gate_row * a.dgate.ld) : row_rsrc(nullptr, 0);
        if (gated) load_gate(gate_row, gate);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float w[V], g[V];
            weight(a.w1, s, w);
            take_gate(gate, s, g);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sw1[s][i] = g[i] * sa[s][i];
                sa[s][i] *= a.alpha * w[i];
            }
            if (a.gate_direct) t.store(dg, s, sa[s]);
        }
    }
    // partial rows, 32 bits each
    float* ws = a.ws + chunk * a.ws_slots * a.ws_pitch;
    auto leave = [&](int slot, float (*v)[V]) {
        if (slot < 0) return;
        const rsrc_t r = row_rsrc(ws + slot * a.ws_pitch, (int)a.ws_pitch * 4);
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < V; i += 4)
                __builtin_amdgcn_raw_buffer_store_b128(
                    (u32x4){as_u(v[s][i]), as_u(v[s][i + 1]), as_u(v[s][i + 2]), as_u(v[s][i + 3])},
                    r, (t.col(s) + i) * 4, 0, 0);
    };
    leave(a.slot_w1, sw1);
    leave(a.slot_w2, sw2);
    leave(a.slot_gate, sa);
}

// Adds partial rows: output row o (blockIdx.y: first dw1 and dw2 as wanted,
// then the gate rows) is the sum over its chunks.  A workgroup takes 64
// columns, 16 lanes of 4, and 64 partial sums of every 64th chunk each, joined
// in the LDS in a fixed order.
constexpr int kJoinCols = 64, kJoinParts = 64;

template <int DT>
__global__ __launch_bounds__(1024) void grad_join_kernel(const GradArgs a, int64_t outputs) {
    __shared__ f32x4 part[kJoinParts][kJoinCols / 4];
    const int lane = (int)threadIdx.x % 16, p = (int)threadIdx.x / 16;
    const int col = (int)blockIdx.x * kJoinCols + lane * 4;
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
        f32x4 sum = (f32x4)(0.0f);
        if (col < a.cols) {
            const float* ws = a.ws + (first * a.ws_slots + slot) * a.ws_pitch + col;
            const int64_t step = (int64_t)a.ws_slots * a.ws_pitch;
#pragma unroll 8
            for (int64_t c = p; c < count; c += kJoinParts)
                sum += *reinterpret_cast<const f32x4*>(ws + c * step);
        }
        part[p][lane] = sum;
        __syncthreads();
#pragma unroll
        for (int half = kJoinParts / 2; half >= 1; half /= 2) {
            if (p < half) part[p][lane] += part[p + half][lane];
            __syncthreads();
        }
        const int c = (int)threadIdx.x, at = (int)blockIdx.x * kJoinCols + c;
        if (c < kJoinCols && at < a.cols) {
            const float total = part[0][c / 4][c % 4];
            if (f32)
                Elem<PTORED_F32>::store1(out + (int64_t)at * 4, total);
            else
                Elem<DT>::store1(out + (int64_t)at * Elem<DT>::kBytes, total);
        }
        __syncthreads();
    }
}

template <int DT, int S, bool PACKED, bool MANY>
static const void* grad_pick(int cols) {
    switch (edge_of<DT>(cols)) {
        case kWhole: return reinterpret_cast<const void*>(grad_kernel<DT, S, kWhole, PACKED, MANY>);
        case kPart: return reinterpret_cast<const void*>(grad_kernel<DT, S, kPart, PACKED, MANY>);
        default: return reinterpret_cast<const void*>(grad_kernel<DT, 1, kTiny, PACKED, MANY>);
    }
}

template <int DT, int S>
static int launch_grad(const GradArgs& a, int threads, hipStream_t stream) {
    const bool packed = a.kx.q != nullptr || a.kh.q != nullptr;
    const bool many = a.gate.p != nullptr && a.chunk_gates > 1;
    const void* k = packed ? (many ? grad_pick<DT, S, true, true>(a.cols)
                                   : grad_pick<DT, S, true, false>(a.cols))
                           : (many ? grad_pick<DT, S, false, true>(a.cols)
                                   : grad_pick<DT, S, false, false>(a.cols));
    void* args[] = {const_cast<GradArgs*>(&a)};
    return hipLaunchKernel(k, dim3((uint32_t)a.chunks), dim3((uint32_t)threads), args, 0,
                           stream) == hipSuccess
               ? kOk
               : kFailed;
}

template <int DT>
int grad_launch(const GradArgs& a, hipStream_t stream) {
    constexpr int V = Elem<DT>::V;
    const int slots = (a.cols + V - 1) / V;
    int per = 1;
    while (slots > per * 1024) per *= 2;
    const int threads = slot_threads(slots, per);
    int rc = kOk;
    if (a.chunks > 0) {
        rc = kFailed;
        if (per == 1) rc = launch_grad<DT, 1>(a, threads, stream);
        if (per == 2) rc = launch_grad<DT, 2>(a, threads, stream);
        if constexpr (V == 4) {
            if (per == 4) rc = launch_grad<DT, 4>(a, threads, stream);
        }
    }
    if (rc != kOk) return rc;
    int64_t outputs = (a.slot_w1 >= 0) + (a.slot_w2 >= 0);
    if (a.slot_gate >= 0) outputs += a.gate_rows;
    if (outputs == 0) return kOk;
    const dim3 grid((uint32_t)((a.cols + kJoinCols - 1) / kJoinCols),
                    (uint32_t)(outputs < 32768 ? outputs : 32768));
    void* args[] = {const_cast<GradArgs*>(&a), &outputs};
    return hipLaunchKernel(reinterpret_cast<const void*>(grad_join_kernel<DT>), grid, dim3(1024),
                           args, 0, stream) == hipSuccess
               ? kOk
               : kFailed;
}

}  // namespace block
}  // namespace ptored
