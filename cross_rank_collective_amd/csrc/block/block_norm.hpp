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
//
// What it took, on one MI355X (bf16, 4096 rows):
//   8 partials of 8192 columns, no norm after the block: 118 us, 6.2 TB/s of
//   the bytes above (112 us at the rate of an elementwise copy).
//   2 partials of 4096 columns, both norms, a gate, h and x' kept in 8 bits:
//   44 us, 4.6 TB/s; four times the rows 141 us, 5.7 TB/s: 8 us of a call are
//   its start and end.  The weights and the gate are asked for before the sum
//   that precedes their use (after it: 47 us).
// One token of 8192 columns and 8 partials takes 3.9 us, of which an empty
// kernel's launch is 1.5 us and the rest one chain of kernel arguments, loads,
// sum and store.
#pragma once

#include "block_device.hpp"

namespace ptored {
namespace block {

// mean(v^2) over the workgroup's row.  The sum of the squares can pass binary32's
// range where the mean does not (at 8192 columns from values of 2e17 on): then
// each square is taken as (v / D) v, whose sum is the mean.  Not always, since
// small values' quotients would lose digits.  Every thread has the same sum, so
// the test is one of scalars.
template <int S, int V>
__device__ __forceinline__ float mean_square(const float (&v)[S][V], float own, float inv_cols,
                                             f32x4 (*red)[1][kMaxWaves / 4], int& turn) {
    float sum[1] = {own};
    block_sum<1>(red[turn], sum);
    turn ^= 1;
    const uint32_t all = (uint32_t)__builtin_amdgcn_readfirstlane((int)as_u(sum[0]));
    if (__builtin_expect(all != 0x7F800000u, 1)) return as_f(all) * inv_cols;
    sum[0] = 0.0f;
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) sum[0] += v[s][i] * inv_cols * v[s][i];
    block_sum<1>(red[turn], sum);
    turn ^= 1;
    return sum[0];
}

// S slots of a row per thread.  KEEP: at least one output in 8 bits.
template <int DT, int S, int EDGE, bool KEEP>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    // ranks whose slots are in flight together
    constexpr int R = 4;
    typedef Slots<DT, S, EDGE> Row;
    __shared__ f32x4 red[2][1][kMaxWaves / 4];
    const Row t(a.cols);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const bool gated = a.gate.p != nullptr;
        const rsrc_t gate_row =
            t.row(gated ? a.gate.p + row / a.rows_per_gate * a.gate.ld : nullptr);
        u32x4 x_raw[S];
        const rsrc_t x_row = t.row(a.x.p + row * a.x.ld);
#pragma unroll
        for (int s = 0; s < S; ++s) x_raw[s] = t.load(x_row, s);
        float h[S][V];
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) h[s][i] = 0.0f;
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
                    for (int i = 0; i < V; ++i) h[s][i] += y[i];
                }
        }
        const auto& b = args_again<NormArgs>();
        float branch = b.alpha;
        // the factors are asked for before the sum is waited for
        typename Row::Weight w[S];
        u32x4 g[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (b.w1 != nullptr) w[s] = t.load_weight(b.w1, b.w_f32, s);
            if (gated) g[s] = t.load(gate_row, s);
        }
        if (b.w1 != nullptr) {
            float own = 0.0f;
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) own += h[s][i] * h[s][i];
            const float r1 = 1.0f / sqrtf(mean_square(h, own, b.inv_cols, red, turn) + b.eps);
            if (b.r1 != nullptr && threadIdx.x == 0) b.r1[row] = r1;
            branch *= r1;
        }
        if (b.h.p) {
            const rsrc_t out = t.row(b.h.p + row * b.h.ld);
#pragma unroll
            for (int s = 0; s < S; ++s) t.store(out, s, h[s]);
        }
        if (KEEP && b.kh.q) {
            const typename Row::KeptRow out = t.kept_row(b.kh, row);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float v[V];
                E::widen(E::narrow(h[s]), v);
                t.store_kept(out, s, v);
            }
        }
        const auto& c = args_again<NormArgs>();
        float x[S][V], own = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float p[V];
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = branch * h[s][i];
            if (c.w1 != nullptr) {
                float v[V];
                t.take_weight(w[s], c.w_f32, c.offset, s, v);
#pragma unroll
                for (int i = 0; i < V; ++i) p[i] *= v[i];
            }
            if (gated) {
                float v[V];
                t.take(g[s], s, v);
#pragma unroll
                for (int i = 0; i < V; ++i) p[i] *= v[i];
            }
            t.take(x_raw[s], s, x[s]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[s][i] = c.beta * x[s][i] + p[i];
                own += x[s][i] * x[s][i];
            }
        }
        if (c.x_out.p) {
            const rsrc_t out = t.row(c.x_out.p + row * c.x_out.ld);
#pragma unroll
            for (int s = 0; s < S; ++s) t.store(out, s, x[s]);
        }
        if (KEEP && c.kx.q) {
            const typename Row::KeptRow out = t.kept_row(c.kx, row);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                float v[V];
                E::widen(E::narrow(x[s]), v);
                t.store_kept(out, s, v);
            }
        }
        const auto& d = args_again<NormArgs>();
        if (d.w2 == nullptr) continue;  // the same for every wave
#pragma unroll
        for (int s = 0; s < S; ++s) w[s] = t.load_weight(d.w2, d.w_f32, s);
        const float r2 = 1.0f / sqrtf(mean_square(x, own, d.inv_cols, red, turn) + d.eps);
        if (d.r2 != nullptr && threadIdx.x == 0) d.r2[row] = r2;
        if (d.z.p == nullptr && !(KEEP && d.kz.q)) continue;
        const rsrc_t z_row = t.row(d.z.p + row * d.z.ld);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            float z[V];
            t.take_weight(w[s], d.w_f32, d.offset, s, z);
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] *= r2 * x[s][i];
            if (d.z.p) t.store(z_row, s, z);
            if (KEEP && d.kz.q) {
                E::widen(E::narrow(z), z);
                t.store_kept(t.kept_row(d.kz, row), s, z);
            }
        }
    }
}

template <int DT, int S, bool KEEP>
static const void* norm_pick(int cols) {
    switch (edge_of<DT>(cols)) {
        case kWhole: return reinterpret_cast<const void*>(norm_kernel<DT, S, kWhole, KEEP>);
        case kPart: return reinterpret_cast<const void*>(norm_kernel<DT, S, kPart, KEEP>);
        default:
            if constexpr (S == 1)
                return reinterpret_cast<const void*>(norm_kernel<DT, 1, kTiny, KEEP>);
            return nullptr;
    }
}

template <int DT, int S>
static int launch_norm(const NormArgs& a, int threads, hipStream_t stream) {
    const bool keep = a.kh.q != nullptr || a.kx.q != nullptr || a.kz.q != nullptr;
    const void* k = keep ? norm_pick<DT, S, true>(a.cols) : norm_pick<DT, S, false>(a.cols);
    // a launch takes fewer than 2^32 threads
    const int64_t most = (int64_t(1) << 31) / threads;
    const int64_t grid = a.rows < most ? a.rows : most;
    void* args[] = {const_cast<NormArgs*>(&a)};
    return hipLaunchKernel(k, dim3((uint32_t)grid), dim3((uint32_t)threads), args, 0, stream) ==
                   hipSuccess
               ? kOk
               : kFailed;
}

template <int DT>
int norm_launch(const NormArgs& a, hipStream_t stream) {
    constexpr int V = Elem<DT>::V;
    const int slots = (a.cols + V - 1) / V;
    // 16 elements a thread (8: 5% slower over large calls, 32: no faster), 8
    // where the rows leave compute units idle anyway (48 rows of 5120: 5.0
    // us, with 16 5.4)
    int per = (a.rows <= 256 ? 8 : 16) / V;
    while (slots > per * 1024) per *= 2;
    const int threads = slot_threads(slots, per);
    if (per == 1) return launch_norm<DT, 1>(a, threads, stream);
    if (per == 2) return launch_norm<DT, 2>(a, threads, stream);
    if constexpr (V == 4) {
        if (per == 4) return launch_norm<DT, 4>(a, threads, stream);
    }
    return kFailed;  // more than PTORED_BLOCK_MAX_COLS columns
}

}  // namespace block
}  // namespace ptored
