// block_device.hpp -- device helpers of the block-boundary kernels: slots of
// a row in registers, wave and workgroup sums, the 8-bit form.
//
// A slot is 16 bytes of activations: V consecutive elements of one row (8 of
// 16 bits, 4 of 32), held as V floats.  Lane l of a workgroup of B threads
// holds slots l, l + B, ...: every wave instruction covers 1 KiB of a row.
// Rows may start at any element and end inside a slot (TAIL): full slots are
// one unaligned 16-byte access, which the hardware serves, the last partial
// one goes element by element.  Nothing past a row's columns is touched.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "block_plan.h"

namespace ptored {
namespace block {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// the same with an element's alignment, for rows that start anywhere
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float as_f(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t as_u(float f) { return __builtin_bit_cast(uint32_t, f); }

// Element types: conversions between 32-bit words and floats.  Rounding to
// an element type is to nearest, ties to even, once per stored value.
template <int DT>
struct Elem;

template <>
struct Elem<PTORED_F32> {
    static constexpr int kBytes = 4, V = 4;
    static __device__ __forceinline__ void widen(u32x4 w, float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = as_f(w[i]);
    }
    static __device__ __forceinline__ u32x4 narrow(const float* v) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = as_u(v[i]);
        return w;
    }
    static __device__ __forceinline__ float load1(const char* p) {
        return *reinterpret_cast<const float*>(p);
    }
    static __device__ __forceinline__ void store1(char* p, float v) {
        *reinterpret_cast<float*>(p) = v;
    }
};

template <>
struct Elem<PTORED_BF16> {
    static constexpr int kBytes = 2, V = 8;
    static __device__ __forceinline__ void widen(u32x4 w, float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = as_f(w[i] << 16);
            v[2 * i + 1] = as_f(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ u32x4 narrow(const float* v) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __builtin_bit_cast(uint32_t, (b2){(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
        return w;
    }
    static __device__ __forceinline__ float load1(const char* p) {
        return as_f((uint32_t) * reinterpret_cast<const uint16_t*>(p) << 16);
    }
    static __device__ __forceinline__ void store1(char* p, float v) {
        *reinterpret_cast<uint16_t*>(p) = __builtin_bit_cast(uint16_t, (__bf16)v);
    }
};

template <>
struct Elem<PTORED_F16> {
    static constexpr int kBytes = 2, V = 8;
    static __device__ __forceinline__ void widen(u32x4 w, float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const h2 p = __builtin_bit_cast(h2, (uint32_t)w[i]);
            v[2 * i] = (float)p[0];
            v[2 * i + 1] = (float)p[1];
        }
    }
    static __device__ __forceinline__ u32x4 narrow(const float* v) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __builtin_bit_cast(uint32_t, (h2){(_Float16)v[2 * i], (_Float16)v[2 * i + 1]});
        return w;
    }
    static __device__ __forceinline__ float load1(const char* p) {
        return (float)*reinterpret_cast<const _Float16*>(p);
    }
    static __device__ __forceinline__ void store1(char* p, float v) {
        *reinterpret_cast<_Float16*>(p) = (_Float16)v;
    }
};

// The slot of V elements at column `col` of a row of `cols` elements starting
// at `row`; elements past the row are 0.
template <int DT, bool TAIL>
__device__ __forceinline__ void load_slot(const char* row, int col, int cols, float* v) {
    using E = Elem<DT>;
    const char* p = row + (int64_t)col * E::kBytes;
    if (!TAIL ? col < cols : col + E::V <= cols) {
        E::widen(*reinterpret_cast<const u32x4_any*>(p), v);
        return;
    }
#pragma unroll
    for (int i = 0; i < E::V; ++i) v[i] = 0.0f;
    if constexpr (TAIL) {
#pragma unroll
        for (int i = 0; i < E::V - 1; ++i)
            if (col + i < cols) v[i] = E::load1(p + i * E::kBytes);
    }
}

template <int DT, bool TAIL>
__device__ __forceinline__ void store_slot(char* row, int col, int cols, const float* v) {
    using E = Elem<DT>;
    char* p = row + (int64_t)col * E::kBytes;
    if (!TAIL ? col < cols : col + E::V <= cols) {
        *reinterpret_cast<u32x4_any*>(p) = E::narrow(v);
        return;
    }
    if constexpr (TAIL) {
#pragma unroll
        for (int i = 0; i < E::V - 1; ++i)
            if (col + i < cols) E::store1(p + i * E::kBytes, v[i]);
    }
}

// V elements of a norm weight (32 bits, or the activations' type) at `col`,
// plus the offset.
template <int DT, bool TAIL>
__device__ __forceinline__ void load_weight(const char* w, int w_f32, float offset, int col,
                                            int cols, float* v) {
    constexpr int V = Elem<DT>::V;
    if (w_f32) {
#pragma unroll
        for (int i = 0; i < V; i += 4) load_slot<PTORED_F32, TAIL>(w, col + i, cols, v + i);
    } else {
        load_slot<DT, TAIL>(w, col, cols, v);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += offset;
}

// ---------------------------------------------------------------- sums

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t u) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, CTRL, 0xF, 0xF, true);
}
constexpr int kDppXor1 = 0xB1;         // lanes 1 0 3 2 of each quad
constexpr int kDppXor2 = 0x4E;         // lanes 2 3 0 1 of each quad
constexpr int kDppHalfMirror = 0x141;  // lane i of 8 takes 7 - i
constexpr int kDppMirror = 0x140;      // lane i of 16 takes 15 - i

// The wave's sum, the same in every lane: four steps inside rows of 16 lanes
// by data-parallel moves, then the four rows' sums read as scalars.  (A
// shuffle through the LDS per step takes several times as long.)
__device__ __forceinline__ float wave_sum(float x) {
    x += as_f(dpp<kDppXor1>(as_u(x)));
    x += as_f(dpp<kDppXor2>(as_u(x)));
    x += as_f(dpp<kDppHalfMirror>(as_u(x)));
    x += as_f(dpp<kDppMirror>(as_u(x)));
    const int i = (int)as_u(x);
    return (as_f((uint32_t)__builtin_amdgcn_readlane(i, 0)) +
            as_f((uint32_t)__builtin_amdgcn_readlane(i, 16))) +
           (as_f((uint32_t)__builtin_amdgcn_readlane(i, 32)) +
            as_f((uint32_t)__builtin_amdgcn_readlane(i, 48)));
}

constexpr int kMaxWaves = 16;  // waves of the largest workgroup

// Sums of K values over the workgroup, in a fixed order.  `red` is one of the
// caller's buffers; the caller alternates between two, so that one barrier
// per sum is enough: a wave writes a buffer again only after the barrier of
// the sum in between, which every wave reaches after it has read this one.
template <int K>
__device__ __forceinline__ void block_sum(float (*red)[kMaxWaves], float* v) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
    const int waves = (int)blockDim.x >> 6;
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) red[k][threadIdx.x >> 6] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float s = 0.0f;
        for (int w = 0; w < waves; ++w) s += red[k][w];
        v[k] = s;
    }
}

// ---------------------------------------------------------------- 8 bits

// 2^n for n in [-126, 127]
__device__ __forceinline__ float power_of_2(int n) { return as_f((uint32_t)(n + 127) << 23); }

// Largest magnitude of a block of 32 elements, as bits, in all its lanes: a
// block is 4 lanes of 8 elements or 8 lanes of 4.  Bit patterns of
// non-negative floats compare like the values, infinities and NaN above all.
template <int V>
__device__ __forceinline__ uint32_t block_amax(const float* v) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, as_u(v[i]) & 0x7FFFFFFFu);
    m = max(m, dpp<kDppXor1>(m));
    m = max(m, dpp<kDppXor2>(m));
    if constexpr (V == 4) m = max(m, dpp<kDppHalfMirror>(m));
    return m;
}

// Packs the slot at `col` of a row; every lane of the wave takes part (slots
// past the row hold zeros and store nothing).  Zeros past a row's end do not
// change its last block's largest magnitude.
template <int V, bool TAIL>
__device__ __forceinline__ void pack_slot(const Kept& k, int64_t row, int col, int cols,
                                          const float* v) {
    const uint32_t top = block_amax<V>(v);
    const bool finite = top < 0x7F800000u;
    // E: the exponent of amax, one more where amax 2^(6-E) would round to 128
    // (127.5 = 64 * 1.1111111b does, ties to even)
    int e = (int)(top >> 23) - 127 + ((top & 0x7FFFFFu) >= 0x7F0000u ? 1 : 0);
    e = min(max(e, -120), 127);
    const float f = power_of_2(6 - e);
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float r = __builtin_rintf(v[i + j] * f);
            const int q = finite ? (int)fminf(fmaxf(r, -127.0f), 127.0f) : 0;
            word |= ((uint32_t)q & 0xFFu) << (8 * j);
        }
        w[i / 4] = word;
    }
    if (col >= cols) return;
    int8_t* q = k.q + row * k.q_ld + col;
    if (!TAIL || col + V <= cols) {
        if constexpr (V == 8)
            *reinterpret_cast<u32x2_any*>(q) = (u32x2){w[0], w[1]};
        else
            *reinterpret_cast<uint32_t __attribute__((aligned(1)))*>(q) = w[0];
    } else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (col + i < cols) q[i] = (int8_t)(w[i / 4] >> (8 * (i % 4)));
    }
    if ((col & (PTORED_CHECKPOINT_BLOCK - 1)) == 0)
        k.s[row * k.s_ld + col / PTORED_CHECKPOINT_BLOCK] =
            finite ? (uint8_t)(e + 127) : (uint8_t)255;
}

// The factor 2^(E-6) of a scale byte; NaN for 255.
__device__ __forceinline__ float scale_factor(uint32_t s) {
    // bytes below 7 are never written; they count as 7 rather than leave the
    // exponent's range
    return s == 255u ? as_f(0x7FC00000u) : as_f((max(s, 7u) - 6u) << 23);
}

template <int V, bool TAIL>
__device__ __forceinline__ void unpack_slot(const Kept& k, int64_t row, int col, int cols,
                                            float* v) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
    if (col >= cols) return;
    const int8_t* q = k.q + row * k.q_ld + col;
    const float f = scale_factor(k.s[row * k.s_ld + col / PTORED_CHECKPOINT_BLOCK]);
    uint32_t w[V / 4] = {};
    if (!TAIL || col + V <= cols) {
        if constexpr (V == 8) {
            const u32x2 u = *reinterpret_cast<const u32x2_any*>(q);
            w[0] = u[0];
            w[1] = u[1];
        } else {
            w[0] = *reinterpret_cast<const uint32_t __attribute__((aligned(1)))*>(q);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (col + i < cols) w[i / 4] |= (uint32_t)(uint8_t)q[i] << (8 * (i % 4));
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (!TAIL || col + i < cols) v[i] = (float)(int8_t)(w[i / 4] >> (8 * (i % 4))) * f;
}

}  // namespace block
}  // namespace ptored
