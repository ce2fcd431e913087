// checkpoint_wgrad.hpp -- a projection's weight gradient from its packed input.
//
//     dw[o, i] = sum_t dy[t, o] x[t, i],   x[t, i] = q 2^(E-6)
//
// A matrix product over the tokens, both operands with the sum's index as the
// slow one.  The values kept are exact in bfloat16, so x enters the matrix
// instructions without loss; so does dy, as one bfloat16 (bf16), the exact
// sum of two (f16) or of three (f32): products are exact and sums in binary32.
//
// A workgroup computes a tile of dw.  Each step stages kStep tokens of both
// operands in the LDS as bfloat16, token-major as they come from memory, and
// reads them with transposing loads (ds_read_b64_tr_b16: 16 lanes fetch 4
// tokens x 16 columns and receive 4 tokens of one column each), which give a
// lane its 8 tokens of one column without a transposed store.  The order of
// tokens within an instruction is that of the loads, the same for both
// operands, so the sum is over all of them.
//
// LDS rows are cut into 64-byte pieces; row t keeps piece c at c ^ (t & 3), so
// that the four rows a transposing load reads at one piece lie in different
// banks.
#pragma once

#include "block_device.hpp"

namespace ptored {
namespace block {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 64;  // tokens staged at a time

template <int DT>
constexpr int planes_of() {
    return DT == PTORED_BF16 ? 1 : DT == PTORED_F16 ? 2 : 3;
}

// 8 elements of dy as words: as loaded, split into bfloat16 planes on the way
// to the LDS.
template <int DT>
struct DyChunk {
    u32x4 w[DT == PTORED_F32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ DyChunk<DT> load_dy(const char* row, int col, int cols, bool in) {
    using E = Elem<DT>;
    DyChunk<DT> c;
    const char* p = row + (int64_t)col * E::kBytes;
    if (in && col + 8 <= cols) {
        c.w[0] = *reinterpret_cast<const u32x4_any*>(p);
        if constexpr (DT == PTORED_F32) c.w[1] = *reinterpret_cast<const u32x4_any*>(p + 16);
        return c;
    }
    uint32_t w[DT == PTORED_F32 ? 8 : 4] = {};
    if (in) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (col + i >= cols) continue;
            if constexpr (DT == PTORED_F32)
                w[i] = reinterpret_cast<const uint32_t*>(p)[i];
            else
                w[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i % 2));
        }
    }
    c.w[0] = (u32x4){w[0], w[1], w[2], w[3]};
    if constexpr (DT == PTORED_F32) c.w[1] = (u32x4){w[4], w[5], w[6], w[7]};
    return c;
}

// Upper halves of two words, lo's first.
__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi) {
    return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// Plane 0 is the value's upper half (truncated, so that it cannot overflow),
// each next plane that of the exact remainder; infinities and NaN are in
// plane 0 alone.
template <int DT>
__device__ __forceinline__ void split_dy(const DyChunk<DT>& c, u32x4* plane) {
    if constexpr (DT == PTORED_BF16) {
        plane[0] = c.w[0];
    } else {
        float v[8];
        if constexpr (DT == PTORED_F32) {
            Elem<DT>::widen(c.w[0], v);
            Elem<DT>::widen(c.w[1], v + 4);
        } else {
            Elem<DT>::widen(c.w[0], v);
        }
#pragma unroll
        for (int k = 0; k < planes_of<DT>(); ++k) {
            uint32_t hi[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t u = as_u(v[i]);
                const bool finite = (u & 0x7F800000u) != 0x7F800000u;
                hi[i] = u & 0xFFFF0000u;
                if (k == 0 && !finite && (u & 0x7FFFFFu) != 0) hi[i] = 0x7FC00000u;
                v[i] = finite ? v[i] - as_f(hi[i]) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) plane[k][i] = upper_halves(hi[2 * i], hi[2 * i + 1]);
        }
    }
}

// 16 packed values of one block and their factor.
struct KeptChunk {
    u32x4 w;
    uint32_t scale;
};

__device__ __forceinline__ KeptChunk load_kept(const Kept& k, int64_t row, int col, int cols,
                                               bool in) {
    KeptChunk c;
    c.w = (u32x4){0, 0, 0, 0};
    c.scale = 127;
    if (!in || col >= cols) return c;
    const int8_t* q = k.q + row * k.q_ld + col;
    c.scale = k.s[row * k.s_ld + col / PTORED_CHECKPOINT_BLOCK];
    if (col + 16 <= cols) {
        c.w = *reinterpret_cast<const u32x4_any*>(q);
    } else {
        uint32_t w[4] = {};
#pragma unroll
        for (int i = 0; i < 15; ++i)
            if (col + i < cols) w[i / 4] |= (uint32_t)(uint8_t)q[i] << (8 * (i % 4));
        c.w = (u32x4){w[0], w[1], w[2], w[3]};
    }
    return c;
}

// The chunk's values as bfloat16 (exact: at most 8 significant bits).
__device__ __forceinline__ void widen_kept(const KeptChunk& c, u32x4* out) {
    const float f = scale_factor(c.scale);
    uint32_t v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = as_u((float)(int8_t)(c.w[i / 4] >> (8 * (i % 4))) * f);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i / 4][i % 4] = upper_halves(v[2 * i], v[2 * i + 1]);
}

// LDS byte offset of 16-byte chunk `c` of row `t`, rows of `row_bytes`.
__device__ __forceinline__ int lds_chunk(int t, int c, int row_bytes) {
    return t * row_bytes + (((c >> 2) ^ (t & 3)) << 6) + ((c & 3) << 4);
}

// The lane's 8 tokens of one column: 32 columns from piece `piece`, the 16
// tokens from `t0`.  Lanes 0-31 take tokens 0-3 and 8-11, the others 4-7 and
// 12-15.
__device__ __forceinline__ b8 read_fragment(const char* tile, int t0, int piece, int row_bytes) {
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const int lane = (int)threadIdx.x & 63;
    const int t = t0 + (lane >> 5) * 4 + ((lane & 15) >> 2);
    const int at = t * row_bytes + ((piece ^ (t & 3)) << 6) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + at));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + at + 8 * row_bytes));
    return __builtin_bit_cast(
        b8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Waves WM x WN, each computing TM x TN blocks of 32 x 32.
template <int DT, int WM, int WN, int TM, int TN>
__global__ __launch_bounds__(WM* WN * 64) void wgrad_kernel(const WgradArgs a) {
    constexpr int kThreads = WM * WN * 64;
    constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
    constexpr int P = planes_of<DT>();
    constexpr int kRowA = BM * 2, kRowB = BN * 2;
    constexpr int kBytesA = kStep * kRowA, kBytesB = kStep * kRowB;
    constexpr int kChunksA = kStep * BM / 8 / kThreads, kChunksB = kStep * BN / 16 / kThreads;
    static_assert(kChunksA * kThreads * 8 == kStep * BM && kChunksB * kThreads * 16 == kStep * BN,
                  "whole chunks per thread");
    __shared__ __attribute__((aligned(128))) char lds[2][P * kBytesA + kBytesB];

    const int tid = (int)threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int tile = (int)(blockIdx.x % (uint32_t)(a.tiles_m * a.tiles_n));
    const int split = (int)(blockIdx.x / (uint32_t)(a.tiles_m * a.tiles_n));
    const int m0 = tile / a.tiles_n * BM, n0 = tile % a.tiles_n * BN;
    const int64_t begin = split * a.rows_per_split;
    const int64_t end = begin + a.rows_per_split < a.rows ? begin + a.rows_per_split : a.rows;

    DyChunk<DT> dy[kChunksA];
    KeptChunk kept[kChunksB];
    auto fetch = [&](int64_t t0) {
#pragma unroll
        for (int c = 0; c < kChunksA; ++c) {
            const int n = c * kThreads + tid, t = n / (BM / 8), col = m0 + n % (BM / 8) * 8;
            dy[c] = load_dy<DT>(a.dy + (t0 + t) * a.dy_ld, col, a.outs, t0 + t < end);
        }
#pragma unroll
        for (int c = 0; c < kChunksB; ++c) {
            const int n = c * kThreads + tid, t = n / (BN / 16), col = n0 + n % (BN / 16) * 16;
            kept[c] = load_kept(a.x, t0 + t, col, a.cols, t0 + t < end);
        }
    };
    auto stage = [&](char* buf) {
#pragma unroll
        for (int c = 0; c < kChunksA; ++c) {
            const int n = c * kThreads + tid, t = n / (BM / 8), at = n % (BM / 8);
            u32x4 plane[P];
            split_dy<DT>(dy[c], plane);
#pragma unroll
            for (int p = 0; p < P; ++p)
                *reinterpret_cast<u32x4*>(buf + p * kBytesA + lds_chunk(t, at, kRowA)) = plane[p];
        }
#pragma unroll
        for (int c = 0; c < kChunksB; ++c) {
            const int n = c * kThreads + tid, t = n / (BN / 16), at = n % (BN / 16) * 2;
            u32x4 v[2];
            widen_kept(kept[c], v);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<u32x4*>(buf + P * kBytesA + lds_chunk(t, at + i, kRowB)) = v[i];
        }
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = (f32x16)(0.0f);
    const int pm = wave / WN * TM, pn = wave % WN * TN;  // the wave's 64-byte pieces

    // One barrier a step: a buffer is written again only after the barrier
    // that every wave reaches once it has read it.
    if (begin < end) {
        fetch(begin);
        stage(lds[0]);
    }
    int cur = 0;
    for (int64_t t0 = begin; t0 < end; t0 += kStep, cur ^= 1) {
        __syncthreads();
        const bool more = t0 + kStep < end;
        if (more) fetch(t0 + kStep);
        const char* buf = lds[cur];
#pragma unroll
        for (int k = 0; k < kStep; k += 16) {
            b8 fb[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j)
                fb[j] = read_fragment(buf + P * kBytesA, k, pn + j, kRowB);
#pragma unroll
            for (int p = 0; p < P; ++p) {
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const b8 fa = read_fragment(buf + p * kBytesA, k, pm + i, kRowA);
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb[j], acc[i][j],
                                                                           0, 0, 0);
                }
            }
        }
        if (more) stage(lds[cur ^ 1]);
    }

    // Register r of a 32 x 32 block is row 8 (r / 4) + 4 (lane / 32) + r % 4,
    // column lane % 32.
    const int64_t ws_ld = a.cols;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int col = n0 + (pn + j) * 32 + (lane & 31);
            if (col >= a.cols) continue;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = m0 + (pm + i) * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
                if (row >= a.outs) continue;
                float v = acc[i][j][r];
                if (a.splits > 1) {
                    a.ws[((int64_t)split * a.outs + row) * ws_ld + col] = v;
                } else if (a.dw_f32) {
                    float* p = reinterpret_cast<float*>(a.dw + row * a.dw_ld) + col;
                    *p = a.accumulate ? *p + v : v;
                } else {
                    char* p = a.dw + row * a.dw_ld + (int64_t)col * Elem<DT>::kBytes;
                    if (a.accumulate) v += Elem<DT>::load1(p);
                    Elem<DT>::store1(p, v);
                }
            }
        }
}

// dw (+)= the splits' sums, in order.  With no token at all, zeros.
constexpr int kJoinThreads = 256;
template <int DT>
__global__ __launch_bounds__(kJoinThreads) void wgrad_join_kernel(const WgradArgs a) {
    const int64_t n = (int64_t)a.outs * a.cols;
    for (int64_t e = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; e < n;
         e += (int64_t)gridDim.x * kJoinThreads) {
        float v = 0.0f;
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) v += a.ws[s * n + e];
        const int64_t row = e / a.cols, col = e - row * a.cols;
        if (a.dw_f32) {
            float* p = reinterpret_cast<float*>(a.dw + row * a.dw_ld) + col;
            *p = a.accumulate ? *p + v : v;
        } else {
            char* p = a.dw + row * a.dw_ld + col * Elem<DT>::kBytes;
            if (a.accumulate) v += Elem<DT>::load1(p);
            Elem<DT>::store1(p, v);
        }
    }
}

template <int DT>
int wgrad_launch(const WgradArgs& a, hipStream_t stream) {
    void* args[] = {const_cast<WgradArgs*>(&a)};
    if (a.splits > 0) {
        const dim3 grid((uint32_t)(a.tiles_m * a.tiles_n) * (uint32_t)a.splits);
        const void* k = reinterpret_cast<const void*>(wgrad_kernel<DT, 2, 2, 2, 2>);
        if (hipLaunchKernel(k, grid, dim3(256), args, 0, stream) != hipSuccess) return kFailed;
    }
    if (a.splits == 1) return kOk;
    const int64_t n = (int64_t)a.outs * a.cols;
    int64_t grid = (n + kJoinThreads - 1) / kJoinThreads;
    if (grid > 65536) grid = 65536;
    return hipLaunchKernel(reinterpret_cast<const void*>(wgrad_join_kernel<DT>),
                           dim3((uint32_t)grid), dim3(kJoinThreads), args, 0,
                           stream) == hipSuccess
               ? kOk
               : kFailed;
}

}  // namespace block
}  // namespace ptored
