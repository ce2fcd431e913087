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
// leaves one partial row per sum in the workspace (A where its rows share one
// gate row, dw1's share where they do not), and a second kernel adds those in a
// fixed order.
//
// What it took, on one MI355X: 16384 x 4096 in bf16 from packed activations
// 112 us (5.9 TB/s of its bytes; 127 us, 5.3 TB/s, call after call, when each
// also pays for the last one's writes) and 6 us for the second kernel; 4096 x
// 1536 in f32 from whole ones 31 + 6.5 us (4.9 TB/s).  A row takes a wave 240
// vector instructions, a third of the time.  Chunks of consecutive rows
// instead of interleaved ones, whose workgroups keep hitting the same memory
// channels, took 136 us for the first; two rows ahead instead of one do not
// fit the registers (187 us).
#pragma once

#include <algorithm>

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

// GATES: with one gate row in the chunk its gradients come from A; a gate row
// for every row needs no A, and saves 12% of what the general form takes (8192
// x 4096 in bf16, packed: 108 us, 122 us).
template <int DT, int S, int EDGE, bool PACKED, int GATES>
__global__ __launch_bounds__(1024) void grad_kernel(const GradArgs a) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    // Up to 8 elements a thread (8192 columns), the factors that rows share are
    // kept and the next row is loaded ahead; with more neither is done.  128
    // registers (1024 threads) hold all that with one gate row, but for f32 past
    // 4096 columns (0 to 4 spill to scratch memory) and packed rows of fewer
    // than 8 elements of 16 bits (16 to 17); with several gate rows 2 to 62
    // spill in 16 bits, and 35 to 88 in f32 past 4096 columns.  8192 x 4096 in
    // bf16, packed: one gate row 63 us, one for each row 105, for every two 123.
    // With more than 8 elements 29 to 183 spill: 2048 x 16384 147 us, 2.3 TB/s.
    constexpr bool HOLD = S * V <= 8;
    constexpr bool MANY = GATES != kOneGate, EACH = GATES == kEachGate;
    typedef Slots<DT, S, EDGE> Row;
    __shared__ f32x4 red[2][3][kMaxWaves / 4];
    const Row t(a.cols);
    const int64_t chunk = blockIdx.x;
    const int64_t unit = chunk / a.chunks_per_unit;
    const int64_t part = chunk - unit * a.chunks_per_unit;
    const int64_t begin = unit * a.unit_rows + part * a.chunk_first;
    const int64_t left = a.unit_rows - part * a.chunk_first;
    const int rows = (int)min(a.chunk_rows, (left + a.row_step - 1) / a.row_step);
    const bool pre = a.w2 != nullptr, post = a.w1 != nullptr, gated = a.gate.p != nullptr;

    // what a row is made of, as loaded; absent rows read as zeros
    struct Raw {
        u32x4 dz[S], dxo[S];
        Activation<PACKED> x[S], h[S];
        float r1, r2;
    };
    // The row's place in a matrix, advanced from row to row.
    struct Place {
        const char* p;
        int64_t ld;
    };
    auto place = [&](const void* p, int64_t ld) -> Place {
        return {static_cast<const char*>(p) + begin * ld, ld * a.row_step};
    };
    const int row_bytes = a.cols * E::kBytes, kept_bytes = PACKED ? a.cols : row_bytes;
    const int blocks = (a.cols + PTORED_CHECKPOINT_BLOCK - 1) / PTORED_CHECKPOINT_BLOCK;
    Place dz = place(a.dz.p, a.dz.ld), dxi = place(a.dxo.p, a.dxo.ld);
    Place x0 = PACKED ? place(a.kx.q, a.kx.q_ld) : place(a.x.p, a.x.ld);
    Place h0 = PACKED ? place(a.kh.q, a.kh.q_ld) : place(a.h.p, a.h.ld);
    Place xs = place(a.kx.s, a.kx.s_ld), hs = place(a.kh.s, a.kh.s_ld);
    Place dxp = place(a.dx.p, a.dx.ld), dhp = place(a.dh.p, a.dh.ld);
    // what there is of them; an absent matrix has rows of no bytes
    enum : uint32_t { kDz = 1, kDxo = 2, kX = 4, kH = 8, kDx = 16, kDh = 32, kRead = 15 };
    uint32_t there = (pre ? kDz | kX : 0) | (a.dxo.p ? kDxo : 0) | (a.dx.p ? kDx : 0) |
                     (a.dh.p ? kDh : 0) |
                     ((PACKED ? a.kh.q != nullptr : a.h.p != nullptr) ? kH : 0);
    auto next_row = [&](Place& m, uint32_t which, int bytes) {
        const rsrc_t r = row_rsrc(m.p, there & which ? bytes : 0);
        m.p += m.ld;
        return r;
    };
    // Loads the next row, or nothing past the chunk's last.
    auto load = [&](int row, Raw& to) {
        if (row >= rows) there &= ~kRead;
        const rsrc_t z = next_row(dz, kDz, row_bytes), d = next_row(dxi, kDxo, row_bytes);
        const rsrc_t x = next_row(x0, kX, kept_bytes), h = next_row(h0, kH, kept_bytes);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            to.dz[s] = t.load(z, s);
            to.dxo[s] = t.load(d, s);
        }
        if constexpr (PACKED) {
            const typename Row::KeptRow kx = {x, next_row(xs, kX, blocks)};
            const typename Row::KeptRow kh = {h, next_row(hs, kH, blocks)};
#pragma unroll
            for (int s = 0; s < S; ++s) {
                to.x[s].w = t.load_kept(kx, s);
                to.h[s].w = t.load_kept(kh, s);
            }
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s) {
                to.x[s].w = t.load(x, s);
                to.h[s].w = t.load(h, s);
            }
        }
        const int64_t at = begin + (row < rows ? row : 0) * a.row_step;
        to.r2 = pre ? a.r2[at] : 0.0f;
        to.r1 = post ? a.r1[at] : 1.0f;
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
    auto take_weight = [&](const typename Row::Weight& raw, const char* w, int s, float* v) {
        t.take_weight(raw, a.w_f32, a.offset, s, v);
        if (w == nullptr) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = 1.0f;
        }
    };
    auto weight = [&](const char* w, int s, float* v) {
        take_weight(t.load_weight(w, a.w_f32, s), w, s, v);
    };
    auto load_gate = [&](int64_t gate_row, u32x4* to) {
        const rsrc_t r = row_rsrc(a.gate.p + gate_row * a.gate.ld, gated ? row_bytes : 0);
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
    // the rows up to here share the gate row
    int64_t gate_end = !MANY ? rows : a.row_step > 1 ? 1 : (gate_row + 1) * a.rows_per_gate - begin;
    u32x4 gate[S];  // of the next row, where that begins a gate row
    load_gate(gate_row, gate);
    // HOLD: w2 + o; alpha g; alpha g (w1 + o), or with MANY w1 + o
    float w2[S][V], ag[S][V], kw[S][V];
    Raw raw;
    if constexpr (HOLD) {
        // everything is asked for before the first wait
        typename Row::Weight w1_raw[S], w2_raw[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            w1_raw[s] = t.load_weight(a.w1, a.w_f32, s);
            w2_raw[s] = t.load_weight(a.w2, a.w_f32, s);
        }
        load(0, raw);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            take_weight(w2_raw[s], a.w2, s, w2[s]);
            take_weight(w1_raw[s], a.w1, s, kw[s]);
            if constexpr (!MANY) {
                take_gate(gate, s, ag[s]);
#pragma unroll
                for (int i = 0; i < V; ++i) kw[s][i] *= ag[s][i];
            }
        }
    }
    u32x4 gate_now[S];  // EACH: of the current row
    // alpha g (w1 + o) of the current row
    auto scale = [&](int s, float* v) {
        if constexpr (HOLD && EACH) {
            take_gate(gate_now, s, v);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= kw[s][i];
        } else if constexpr (!HOLD) {
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
    bool fresh = MANY;  // the row begins a gate row, or the chunk
    auto one_row = [&](int row, Raw& raw, Raw& next) {
        if constexpr (!HOLD) {
            load(row, raw);
            if (MANY && fresh) load_gate(gate_row, gate);
        }
        if constexpr (HOLD && EACH) {
#pragma unroll
            for (int s = 0; s < S; ++s) gate_now[s] = gate[s];
        } else if (HOLD && MANY && fresh) {
#pragma unroll
            for (int s = 0; s < S; ++s) take_gate(gate, s, ag[s]);
        }
        const float r1 = raw.r1, r2 = raw.r2;
        float dxo[S][V], xh[S][V], hh[S][V];
        float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float u[V], k[V];
            t.take(raw.dz[s], s, u);
            t.take(raw.dxo[s], s, dxo[s]);
            take(raw.x[s], s, r2, xh[s]);
            take(raw.h[s], s, r1, hh[s]);
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
        if constexpr (HOLD) {
            load(row + 1, next);
            if ((EACH || fresh) && row + 1 < rows) load_gate(gate_row + a.row_step, gate);
        }
        if (post || pre) block_sum<3>(red[turn], sum);
        turn ^= 1;
        const float c2 = r2 * sum[0] * a.inv_cols;
        const float c1 = r1 * ((sum[1] - c2 * sum[2]) * a.inv_cols);
        const rsrc_t dh_row = next_row(dhp, kDh, row_bytes), dx_row = next_row(dxp, kDx, row_bytes);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float dh[V], k[V];
            scale(s, k);
            float now[V];  // MANY: alpha g
            if constexpr (EACH && HOLD) {
                take_gate(gate_now, s, now);
            } else if constexpr (MANY && !HOLD) {
                take_gate(gate, s, now);
            } else if constexpr (MANY) {
#pragma unroll
                for (int i = 0; i < V; ++i) now[i] = ag[s][i];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = dxo[s][i] - xh[s][i] * c2;  // s
                const float e = d * hh[s][i];
                if constexpr (EACH)
                    sa[s][i] = e;
                else
                    sa[s][i] += e;
                if constexpr (MANY) sw1[s][i] += now[i] * e;
                dh[i] = r1 * (k[i] * d);
                dxo[s][i] = a.beta * d;
            }
            if (post) {
#pragma unroll
                for (int i = 0; i < V; ++i) dh[i] -= hh[s][i] * c1;
            }
            t.store(dh_row, s, dh);
            t.store(dx_row, s, dxo[s]);
        }
        if (MANY && (EACH || fresh || row + 1 == rows)) {
            if (a.gate_direct) {
                const rsrc_t r = t.row(a.dgate.p + gate_row * a.dgate.ld);
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    float w[V];
                    if constexpr (!HOLD) weight(a.w1, s, w);
#pragma unroll
                    for (int i = 0; i < V; ++i) sa[s][i] *= a.alpha * (HOLD ? kw[s][i] : w[i]);
                    t.store(r, s, sa[s]);
                }
            }
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) sa[s][i] = 0.0f;
            gate_row += a.row_step;
            gate_end += a.row_step > 1 ? 1 : a.rows_per_gate;
        }
    };
    // two rows a turn, each loading the other's: nothing is copied between them
    Raw other;
    for (int row = 0; row < rows; row += 2) {
        one_row(row, raw, other);
        if (row + 1 == rows) break;
        one_row(row + 1, other, raw);
    }
    // the arguments read again: nothing that only this end needs stays in
    // registers over the rows
    const auto& z = args_again<GradArgs>();
    // partial rows, 32 bits each
    float* ws = z.ws + chunk * z.ws_slots * z.ws_pitch;
    auto leave = [&](int slot, float (*v)[V]) {
        if (slot < 0) return;
        const rsrc_t r = row_rsrc(ws + slot * z.ws_pitch, (int)z.ws_pitch * 4);
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < V; i += 4)
                __builtin_amdgcn_raw_buffer_store_b128(
                    (u32x4){as_u(v[s][i]), as_u(v[s][i + 1]), as_u(v[s][i + 2]), as_u(v[s][i + 3])},
                    r, (t.col(s) + i) * 4, 0, 0);
    };
    leave(z.slot_w1, MANY ? sw1 : sa);
    leave(z.slot_w2, sw2);
}

// Adds partial rows: output row o (blockIdx.y: first dw1 and dw2 as wanted,
// then the gate rows) is the sum over its chunks, dw1's times their gate rows.
// A workgroup takes COLS columns in lanes of 4 and 4096 / COLS partial sums, one
// for each chunk of a stride, joined in the LDS in a fixed order.  64 columns
// (512 chunks of 4096 columns: 6.5 us; with 32 8.9, with 128 7.5) where that
// makes more than 112 workgroups.  Below it compute units idle, and 32 take
// less time (3500 columns of two weights, 768 chunks: 6.4 us against 7.2, with 16
// 9.7; four rows of 747: 11.5, 21.6 and 14.3), at no more than 32 workgroups 16
// (1000 columns of a weight: 6.7 us, with 32 8.2, with 64 10.1).

// Gate rows of no more than kFlatChunks chunks, in more workgroups than the chip
// holds at once (two a compute unit): there the last `flat` rows of workgroups
// take 4 columns of a gate row for every thread instead (4096 x 4096 with 128
// gate rows 65 -> 9 us, with 32 20 -> 8.5 us; with 8, which fit, 8.6 and 9; 8
// rows of 1024 columns 4.7 and 7.8).
constexpr int kFlatChunks = 32;

template <int DT, int COLS>
__global__ __launch_bounds__(1024) void grad_join_kernel(const GradArgs a, int64_t outputs,
                                                         uint32_t flat) {
    using E = Elem<DT>;
    // alpha (w1 + o) A
    auto gate_gradient = [&](float sum, int at) {
        sum *= a.alpha;
        if (a.w1 != nullptr)
            sum *= a.offset + (a.w_f32 ? Elem<PTORED_F32>::load1(a.w1 + (int64_t)at * 4)
                                       : E::load1(a.w1 + (int64_t)at * E::kBytes));
        return sum;
    };
    if (blockIdx.y >= gridDim.y - flat) {
        const int64_t quads = a.ws_pitch / 4, items = a.gate_rows * quads;
        const int64_t block = (int64_t)(blockIdx.y - (gridDim.y - flat)) * gridDim.x + blockIdx.x;
        const int64_t stride = (int64_t)a.ws_slots * a.ws_pitch;
        for (int64_t i = block * 1024 + threadIdx.x; i < items;
             i += (int64_t)flat * gridDim.x * 1024) {
            const int64_t row = i / quads;
            const int at = (int)(i - row * quads) * 4;
            const float* ws = a.ws + row * a.chunks_per_unit * stride + a.slot_w1 * a.ws_pitch + at;
            f32x4 sum = (f32x4)(0.0f);
#pragma unroll 8
            for (int64_t c = 0; c < a.chunks_per_unit; ++c)
                sum += *reinterpret_cast<const f32x4*>(ws + c * stride);
            char* out = a.dgate.p + row * a.dgate.ld;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (at + k < a.cols)
                    E::store1(out + (int64_t)(at + k) * E::kBytes, gate_gradient(sum[k], at + k));
        }
        return;
    }
    constexpr int kLanes = COLS / 4, kParts = 1024 / kLanes;
    __shared__ f32x4 part[kParts][kLanes];
    const int lane = (int)threadIdx.x % kLanes, p = (int)threadIdx.x / kLanes;
    const int col = (int)blockIdx.x * COLS + lane * 4;
    const int weights = (a.dw1 != nullptr) + (a.dw2 != nullptr);
    // the gate's values at this thread's columns (zeros past the row)
    auto gate_factors = [&](const char* row) {
        const char* q = row + (int64_t)col * E::kBytes;
        f32x4 g = (f32x4)(0.0f);
        if constexpr (E::V == 4) {
            if (col + 4 <= a.cols) return __builtin_bit_cast(f32x4, (u32x4)*reinterpret_cast<const u32x4_any*>(q));
        } else {
            if (col + 4 <= a.cols) {
                const u32x2 w = *reinterpret_cast<const u32x2_any*>(q);
                float v[8];
                E::widen((u32x4){w[0], w[1], 0u, 0u}, v);
                return (f32x4){v[0], v[1], v[2], v[3]};
            }
        }
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (col + i < a.cols) g[i] = E::load1(q + i * E::kBytes);
        return g;
    };
    for (int64_t o = blockIdx.y; o < outputs; o += gridDim.y - flat) {
        int slot = a.slot_w1;
        int64_t first = 0, count = a.chunks;
        char* out;
        bool f32 = true, gates = false;
        if (o < weights) {
            const bool is_w1 = a.dw1 != nullptr && o == 0;
            if (!is_w1) slot = a.slot_w2;
            gates = is_w1 && a.chunk_gates == kOneGate;
            out = is_w1 ? a.dw1 : a.dw2;
            f32 = a.w_f32 != 0;
        } else {
            count = a.chunks_per_unit;
            first = (o - weights) * count;
            out = a.dgate.p + (o - weights) * a.dgate.ld;
            f32 = DT == PTORED_F32;
        }
        f32x4 sum = (f32x4)(0.0f);
        if (col < a.cols) {
            const float* ws = a.ws + (first * a.ws_slots + slot) * a.ws_pitch + col;
            const int64_t step = (int64_t)a.ws_slots * a.ws_pitch;
            if (gates && a.gate_units != 0) {
                // each chunk's A times the gate row of its rows
#pragma unroll(COLS == 64 ? 4 : 8)
                for (uint32_t c = (uint32_t)p; c < (uint32_t)count; c += kParts) {
                    const int64_t row = c / (uint32_t)a.chunks_per_unit;
                    sum += *reinterpret_cast<const f32x4*>(ws + c * step) *
                           gate_factors(a.gate.p + row * a.gate.ld);
                }
            } else {
#pragma unroll 8
                for (int64_t c = p; c < count; c += kParts)
                    sum += *reinterpret_cast<const f32x4*>(ws + c * step);
            }
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
            float total = part[0][c / 4][c % 4];
            if (gates) {
                total *= a.alpha;
                if (a.gate.p != nullptr && a.gate_units == 0)  // one gate row for all
                    total *= E::load1(a.gate.p + (int64_t)at * E::kBytes);
            }
            if (o >= weights) total = gate_gradient(total, at);
            if (f32)
                Elem<PTORED_F32>::store1(out + (int64_t)at * 4, total);
            else
                Elem<DT>::store1(out + (int64_t)at * Elem<DT>::kBytes, total);
        }
        __syncthreads();
    }
}

template <int DT, int S, bool PACKED, int GATES>
static const void* grad_pick(int cols) {
    switch (edge_of<DT>(cols)) {
        case kWhole: return reinterpret_cast<const void*>(grad_kernel<DT, S, kWhole, PACKED, GATES>);
        case kPart: return reinterpret_cast<const void*>(grad_kernel<DT, S, kPart, PACKED, GATES>);
        default: return reinterpret_cast<const void*>(grad_kernel<DT, 1, kTiny, PACKED, GATES>);
    }
}

template <int DT, int S>
static int launch_grad(const GradArgs& a, int threads, hipStream_t stream) {
    const bool packed = a.kx.q != nullptr || a.kh.q != nullptr;
    const int gates = a.gate.p == nullptr ? kOneGate : a.chunk_gates;
    const void* k = nullptr;
    switch (gates) {
        case kOneGate:
            k = packed ? grad_pick<DT, S, true, kOneGate>(a.cols)
                       : grad_pick<DT, S, false, kOneGate>(a.cols);
            break;
        case kEachGate:
            k = packed ? grad_pick<DT, S, true, kEachGate>(a.cols)
                       : grad_pick<DT, S, false, kEachGate>(a.cols);
            break;
        default:
            k = packed ? grad_pick<DT, S, true, kSomeGates>(a.cols)
                       : grad_pick<DT, S, false, kSomeGates>(a.cols);
    }
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
    int64_t outputs = (a.dw1 != nullptr) + (a.dw2 != nullptr);
    const bool few = a.gate_joined && a.rows > 0 && a.chunks_per_unit <= kFlatChunks &&
                     a.gate_rows * ((a.cols + 63) / 64) > 512;
    if (a.gate_joined && !few) outputs += a.gate_rows;
    if (outputs == 0 && !few) return kOk;
    const int64_t chunks = few ? a.chunks : a.chunks_per_unit;  // of an output, or of most
    const int64_t groups = chunks > 64 ? (a.cols + 63) / 64 * outputs : 256;
    const int cols = groups <= 32 ? 16 : groups <= 112 ? 32 : 64;
    const void* k = cols == 16   ? reinterpret_cast<const void*>(grad_join_kernel<DT, 16>)
                    : cols == 32 ? reinterpret_cast<const void*>(grad_join_kernel<DT, 32>)
                                 : reinterpret_cast<const void*>(grad_join_kernel<DT, 64>);
    const uint32_t x = (uint32_t)((a.cols + cols - 1) / cols);
    const int64_t per_row = 1024 * (int64_t)x, items = few ? a.gate_rows * (a.ws_pitch / 4) : 0;
    uint32_t flat = (uint32_t)std::min<int64_t>((items + per_row - 1) / per_row, 32768);
    const dim3 grid(x, (uint32_t)(outputs < 32768 ? outputs : 32768) + flat);
    void* args[] = {const_cast<GradArgs*>(&a), &outputs, &flat};
    return hipLaunchKernel(k, grid, dim3(1024), args, 0, stream) == hipSuccess ? kOk : kFailed;
}

}  // namespace block
}  // namespace ptored
