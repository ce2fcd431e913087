// few.hpp -- the gated feed-forward block of few tokens (decoding).
//
//     g = x Wg^T,  u = x Wu^T,  y = f(g) u
//
// Bound by memory: both weights are read once.  They go from memory straight
// into the matrix instructions' registers: a lane's 16 bytes of one feature's
// row are its operand, and the tokens, padded to blocks of 16, are the other
// one, so that nothing passes through the LDS on the way.  A workgroup takes 16
// FB features; its W waves take the columns in turn, units of U steps of 64
// bytes, the next unit's loads in flight while one is multiplied, and add their
// sums in the LDS at the end, in a fixed order.  Where few features leave compute
// units idle, several workgroups share the columns and a second kernel joins them.
//
// Measured: 1 token, 4096 columns, 2 x 8192 features, bf16 25 us, 5.4 TB/s (21.7 at
// the rate of a large copy).  All workgroups at the same column ask the same
// memory channels: each begins at one of its own (252 MB of weights 57 us, rotated
// and with the caches' usual policy 44).  8 waves where 16 are not needed to fill
// the chip (4096 x 8192 29.6, 24.7).
#pragma once

#include "gated.hpp"

namespace ptored {
namespace step {

using namespace block;

typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

// 16 rows of a times 16 rows of b, 64 bytes of each: lane l has 16 bytes of row
// l % 16 from k = V (l / 16) on.
template <int DT>
__device__ __forceinline__ f32x4 multiply16(u32x4 a, u32x4 b, f32x4 acc) {
    if constexpr (DT == PTORED_BF16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a),
                                                       __builtin_bit_cast(b8, b), acc, 0, 0, 0);
    } else if constexpr (DT == PTORED_F16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a),
                                                      __builtin_bit_cast(h8, b), acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(as_f(a[j]), as_f(b[j]), acc, 0, 0, 0);
        return acc;
    }
}

// Tokens in TB blocks of 16.  The columns fill at least one lane's 16 bytes.
//
// ODD: some row of a 16-bit type begins between two words.  16 bytes that begin
// there take two and a half times as long to load, so a lane loads the four words
// from the one on that its 16 bytes begin in, and takes the fifth from the next
// lane; only a unit's last lanes load it (13 tokens x 2545 x 4425 bf16, us: 38 with
// misaligned loads, 25 with five words a lane, 18 so; in rows of 2546 elements 15).
// Of the first and the last of a row's words half may be a neighbour's: it is
// shifted out.
template <int DT, int W, int FB, int TB, int U, bool ODD>
__global__ __launch_bounds__(W * 64) void few_kernel(const ProductArgs a) {
    using E = Elem<DT>;
    constexpr int ES = E::kBytes, V = E::V, kStep = 64 / ES, kUnit = U * kStep;
    __shared__ f32x4 part[W][FB * 2 * TB][64];
    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t f0 = (int64_t)blockIdx.x * (16 * FB);
    const int features = (int)min(a.n - f0, (int64_t)(16 * FB)), tokens = (int)a.m, k = (int)a.k;
    // resources that end with the last row; rows past it are nowhere
    constexpr int kNone = (int)0x80000000u;
    const char *pg = a.b[0] + f0 * a.b_ld[0], *pu = a.b[1] + f0 * a.b_ld[1], *px = a.a[0];
    const int ng = (int)((features - 1) * a.b_ld[0] + k * ES);
    const int nu = (int)((features - 1) * a.b_ld[1] + k * ES);
    const int nx = (int)((tokens - 1) * a.a_ld[0] + k * ES);
    const int col = (lane >> 4) * 16;  // bytes
    int og[FB], ou[FB], ox[TB];
#pragma unroll
    for (int i = 0; i < FB; ++i) {
        const int row = i * 16 + (lane & 15);
        og[i] = row < features ? row * (int)a.b_ld[0] + col : kNone;
        ou[i] = row < features ? row * (int)a.b_ld[1] + col : kNone;
    }
#pragma unroll
    for (int i = 0; i < TB; ++i) {
        const int row = i * 16 + (lane & 15);
        ox[i] = row < tokens ? row * (int)a.a_ld[0] + col : kNone;
    }
    struct Unit {
        u32x4 g[U][FB], u[U][FB], x[U][TB];
        uint32_t g4[FB], u4[FB], x4[TB];  // ODD: the words behind, for the rows' last lanes
    };
    // bytes from the beginning of the word that a matrix's first element lies in; a
    // lane's first word and how many bytes of it are others'
    const auto before = [](const char* p) { return ODD ? (int)(reinterpret_cast<uint64_t>(p) & 2) : 0; };
    const int bg = before(pg), bu = before(pu), bx = before(px);
    int wg[FB], wu[FB], wx[TB], sg[FB], su[FB], sx[TB];
    auto words = [&](int off, int b, int& word, int& shift) {
        shift = off == kNone ? 0 : (off + b) & 2;
        word = off == kNone ? kNone : off + b - shift;
    };
#pragma unroll
    for (int i = 0; i < FB; ++i) {
        words(og[i], bg, wg[i], sg[i]);
        words(ou[i], bu, wu[i], su[i]);
    }
#pragma unroll
    for (int i = 0; i < TB; ++i) words(ox[i], bx, wx[i], sx[i]);
    auto to_words = [](int bytes, int b) { return ODD ? (bytes + b + 3) & ~3 : bytes; };
    // Step s of a unit's chunks, `by` bytes on: the fifth word is the first of the lane
    // 16 on, or of the row's first lane in the next step.
    const int behind = ((lane + 16) & 63) * 4;
    auto shifted = [&](auto& v, const auto& end, int s, int i, int by) -> u32x4 {
        if constexpr (!ODD) return v[s][i];
        const u32x4 w = v[s][i];
        uint32_t first = w[0];
        if (s + 1 < U) first = lane < 16 ? v[s + 1 < U ? s + 1 : s][i][0] : first;
        uint32_t last = (uint32_t)__builtin_amdgcn_ds_bpermute(behind, (int)first);
        if (s + 1 == U) last = lane < 48 ? last : end[i];
        return (u32x4){__builtin_amdgcn_alignbyte(w[1], w[0], by), __builtin_amdgcn_alignbyte(w[2], w[1], by),
                       __builtin_amdgcn_alignbyte(w[3], w[2], by), __builtin_amdgcn_alignbyte(last, w[3], by)};
    };
    Unit one, two;
    // units without an end in them; this split's among them
    const int split = (int)blockIdx.y, units = k / kUnit;
    const int first = (int)((int64_t)units * split / a.splits);
    const int whole = (int)((int64_t)units * (split + 1) / a.splits) - first;
    // Each workgroup begins at a unit of its own: the rows of all of them are a
    // pitch apart, and at one column they would ask the same memory channels.
    const int turn = whole > 0 ? (int)((uint32_t)blockIdx.x * W % (uint32_t)whole) : 0;
    // Past the last unit the resources are empty: zeros without a branch, which
    // would have every wait count on the way without loads.
    auto load = [&](Unit& to, int unit) {
        const bool in = unit < whole;
        const int from = (first + (unit + turn < whole ? unit + turn : unit + turn - whole)) * (U * 64);
        const rsrc_t rg = row_rsrc(pg - bg, in ? to_words(ng, bg) : 0);
        const rsrc_t ru = row_rsrc(pu - bu, in ? to_words(nu, bu) : 0);
        const rsrc_t rx = row_rsrc(px - bx, in ? to_words(nx, bx) : 0);
#pragma unroll
        for (int s = 0; s < U; ++s) {
#pragma unroll
            for (int i = 0; i < FB; ++i) {
                to.g[s][i] = __builtin_amdgcn_raw_buffer_load_b128(rg, wg[i], from + s * 64, kPolicyKeep);
                to.u[s][i] = __builtin_amdgcn_raw_buffer_load_b128(ru, wu[i], from + s * 64, kPolicyKeep);
            }
#pragma unroll
            for (int i = 0; i < TB; ++i)
                to.x[s][i] = __builtin_amdgcn_raw_buffer_load_b128(rx, wx[i], from + s * 64, kPolicyKeep);
        }
        if constexpr (ODD) {
            const int end = from + U * 64 - 48;
            auto word = [&](rsrc_t r, int off) {
                return __builtin_amdgcn_raw_buffer_load_b32(r, lane < 48 ? kNone : off, end, kPolicyKeep);
            };
#pragma unroll
            for (int i = 0; i < FB; ++i) {
                to.g4[i] = word(rg, wg[i]);
                to.u4[i] = word(ru, wu[i]);
            }
#pragma unroll
            for (int i = 0; i < TB; ++i) to.x4[i] = word(rx, wx[i]);
        }
    };
    f32x4 ag[FB][TB], au[FB][TB];
#pragma unroll
    for (int i = 0; i < FB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) ag[i][j] = au[i][j] = (f32x4)(0.0f);
    auto multiply = [&](const Unit& v) {
#pragma unroll
        for (int s = 0; s < U; ++s) {
#pragma unroll
            for (int j = 0; j < TB; ++j) {
                const u32x4 x = shifted(v.x, v.x4, s, j, sx[j]);
#pragma unroll
                for (int i = 0; i < FB; ++i) {
                    ag[i][j] = multiply16<DT>(shifted(v.g, v.g4, s, i, sg[i]), x, ag[i][j]);
                    au[i][j] = multiply16<DT>(shifted(v.u, v.u4, s, i, su[i]), x, au[i][j]);
                }
            }
        }
    };
    // What the units leave, at most U steps, is taken first, a step by each of the
    // first waves.  A chunk that the rows' end cuts is loaded so that it ends with
    // them, and moved.
    static_assert(U <= W, "a wave for each step that is left");
    const int rest = split + 1 == a.splits ? units * kUnit + wave * kStep : k;
    u32x4 tg[FB], tu[FB], tx[TB];
    int by = 0;
    if (rest < k) {
        const int at = rest + (lane >> 4) * V;
        by = at < k ? max(at + V - k, 0) : 0;
        auto ending = [&](const char* p, int bytes, int off) {
            return __builtin_amdgcn_raw_buffer_load_b128(
                row_rsrc(p, bytes), at < k && off != kNone ? off + (rest - by) * ES : kNone, 0, 0);
        };
#pragma unroll
        for (int i = 0; i < FB; ++i) {
            tg[i] = ending(pg, ng, og[i]);
            tu[i] = ending(pu, nu, ou[i]);
        }
#pragma unroll
        for (int j = 0; j < TB; ++j) tx[j] = ending(px, nx, ox[j]);
    }
    load(one, wave);
    if (rest < k) {
#pragma unroll
        for (int j = 0; j < TB; ++j) tx[j] = shift_down(tx[j], by * ES);
#pragma unroll
        for (int i = 0; i < FB; ++i) {
            tg[i] = shift_down(tg[i], by * ES);
            tu[i] = shift_down(tu[i], by * ES);
#pragma unroll
            for (int j = 0; j < TB; ++j) {
                ag[i][j] = multiply16<DT>(tg[i], tx[j], ag[i][j]);
                au[i][j] = multiply16<DT>(tu[i], tx[j], au[i][j]);
            }
        }
    }
    for (int unit = wave; unit < whole; unit += 2 * W) {
        load(two, unit + W);
        __builtin_amdgcn_sched_barrier(0);  // or the products are moved before the loads
        multiply(one);
        __builtin_amdgcn_sched_barrier(0);
        load(one, unit + 2 * W);
        __builtin_amdgcn_sched_barrier(0);
        multiply(two);
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < FB; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) {
            part[wave][(i * TB + j) * 2][lane] = ag[i][j];
            part[wave][(i * TB + j) * 2 + 1][lane] = au[i][j];
        }
    __syncthreads();
    // Register r of a lane's sum: feature 4 (lane / 16) + r, token lane % 16.
    // Consecutive threads take consecutive features.
    for (int o = (int)threadIdx.x; o < FB * TB * 256; o += W * 64) {
        const int f = o % (16 * FB), t = o / (16 * FB);
        const int block = (f / 16 * TB + t / 16) * 2, from = (f % 16 / 4) * 16 + t % 16, r = f % 4;
        if (f >= features || t >= tokens) continue;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            g += part[w][block][from][r];
            u += part[w][block + 1][from][r];
        }
        if (a.splits > 1) {
            float* to = a.ws + ((int64_t)split * 2 * tokens + t) * a.ws_ld + f0 + f;
            to[0] = g;
            to[tokens * a.ws_ld] = u;
            continue;
        }
        const int64_t at = (f0 + f) * ES;
        E::store1(a.out[0].p + t * a.out[0].ld + at, activation<DT>(a.activation, g) * u);
        if (a.gate.p) E::store1(a.gate.p + t * a.gate.ld + at, g);
        if (a.up.p) E::store1(a.up.p + t * a.up.ld + at, u);
    }
}

template <int DT, int FB, int TB, int U>
static const void* few_pick(const ProductArgs& a, int& threads) {
    threads = 512;
    if constexpr (FB == 1 && TB == 1) {
        if constexpr (DT != PTORED_F32) {
            uint64_t at = reinterpret_cast<uint64_t>(a.a[0]) | (a.m > 1 ? (uint64_t)a.a_ld[0] : 0);
            for (int i = 0; i < 2; ++i) at |= reinterpret_cast<uint64_t>(a.b[i]) | (uint64_t)a.b_ld[i];
            // (16 waves leave no registers for the fifth words)
            if (at & 2) return reinterpret_cast<const void*>(few_kernel<DT, 8, FB, TB, U, true>);
        }
        if (a.waves == 16) {
            threads = 1024;
            return reinterpret_cast<const void*>(few_kernel<DT, 16, FB, TB, U, false>);
        }
    }
    return reinterpret_cast<const void*>(few_kernel<DT, 8, FB, TB, U, false>);
}

template <int DT>
int few_launch(const ProductArgs& a, hipStream_t stream) {
    int threads = 0;
    const void* k;
    if (a.shape == kFew16)
        k = few_pick<DT, 1, 1, 4>(a, threads);
    else if constexpr (DT != PTORED_F32)
        return kFailed;
    else
        k = a.shape == kFew32 ? few_pick<DT, 1, 2, 4>(a, threads) : few_pick<DT, 2, 4, 2>(a, threads);
    void* args[] = {const_cast<ProductArgs*>(&a)};
    return hipLaunchKernel(k, dim3((uint32_t)a.tiles_n, (uint32_t)a.splits), dim3((uint32_t)threads), args, 0,
                           stream) == hipSuccess
               ? kOk
               : kFailed;
}

}  // namespace step
}  // namespace ptored
