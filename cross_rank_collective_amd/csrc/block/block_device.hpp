// block_device.hpp -- device helpers of the block-boundary kernels: slots of
// a row in registers, wave and workgroup sums, the 8-bit form.
//
// A slot is 16 bytes of activations: V consecutive elements of one row (8 of
// 16 bits, 4 of 32), held as V floats.  Thread l of a workgroup of B holds
// slots l, l + B, ..., S of them: every wave instruction covers 1 KiB of a
// row.  Rows are accessed through buffer resources that end with the row, so
// slots past it read as zeros and are not stored without a branch.  Rows may
// start at any element (the hardware serves unaligned accesses) and end
// inside a slot (EDGE).
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
typedef uint32_t u32_any __attribute__((aligned(1)));
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

// ---------------------------------------------------------------- rows

typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr int kPolicyStream = 2;  // nt: read once
// sc1: written through at device scope (f32 gradients of 4096 x 1536 31 us, with
// nt 33 us; others the same or up to 4% faster)
constexpr int kPolicyStore = 16;
constexpr int kPolicyKeep = 0;    // weights, which every row reads

__device__ __forceinline__ rsrc_t row_rsrc(const void* base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}

// The 16 bytes of `v` without the first `n` (0 to 15), zeros behind.
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int n) {
    const bool two = n & 8, one = n & 4;
    v = (u32x4){two ? v[2] : v[0], two ? v[3] : v[1], two ? 0u : v[2], two ? 0u : v[3]};
    v = (u32x4){one ? v[1] : v[0], one ? v[2] : v[1], one ? v[3] : v[2], one ? 0u : v[3]};
    const uint32_t b = (uint32_t)n & 3u;
    return (u32x4){__builtin_amdgcn_alignbyte(v[1], v[0], b),
                   __builtin_amdgcn_alignbyte(v[2], v[1], b),
                   __builtin_amdgcn_alignbyte(v[3], v[2], b),
                   __builtin_amdgcn_alignbyte(0u, v[3], b)};
}

// The same for 8 words and whole words.
__device__ __forceinline__ void shift_words(uint32_t* w, int n) {
#pragma unroll
    for (int b = 4; b >= 1; b /= 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = n & b ? (i + b < 8 ? w[i + b] : 0u) : w[i];
    }
}

// Rows that end inside a slot.
enum : int {
    kWhole = 0,  // they do not
    kPart = 1,   // the last slot is loaded so that it ends with the row, and moved
    kTiny = 2,   // rows shorter than a slot: element by element
};
template <int DT>
inline int edge_of(int cols) {
    constexpr int V = Elem<DT>::V;
    return cols % V == 0 ? kWhole : cols > V ? kPart : kTiny;
}

// The kernel's arguments, through a pointer that the compiler cannot tell from
// another, so that it loads them where they are used and keeps none of them in
// scalar registers until then.
template <typename A>
__device__ __forceinline__ const A& args_again() {
    typedef const __attribute__((address_space(4))) A* constant_ptr;
    auto p = (constant_ptr)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const A*)p;
}

// A packed slot as loaded: V values and their block's scale byte.
struct KeptRaw {
    u32x2 q;
    uint32_t scale;
};

// Where this thread's S slots lie in a row of `cols` elements.  The launch
// has S - 1 slots of every thread inside the row: only the last can lie past
// it or be cut by its end.
template <int DT, int S, int EDGE>
struct Slots {
    using E = Elem<DT>;
    static constexpr int V = E::V, ES = E::kBytes;
    int cols, stride;  // elements
    int col0, last;    // column of the first slot, and of the last as loaded
    int lost;          // elements of the last, as loaded, that belong to the one before
    bool part;

    __device__ __forceinline__ explicit Slots(int n) {
        cols = n;
        stride = (int)blockDim.x * V;
        col0 = (int)threadIdx.x * V;
        last = col(S - 1);
        part = EDGE != kWhole && last < cols && last + V > cols;
        lost = 0;
        if (EDGE == kPart && part) {
            lost = last + V - cols;
            last = cols - V;
        }
    }
    __device__ __forceinline__ int col(int s) const { return col0 + s * stride; }
    __device__ __forceinline__ int at(int s) const { return s == S - 1 ? last : col(s); }
    __device__ __forceinline__ rsrc_t row(const char* p) const { return row_rsrc(p, cols * ES); }

    // The slot as loaded, to be passed to take() when it is used.
    __device__ __forceinline__ u32x4 load(rsrc_t r, int s) const {
        if constexpr (EDGE == kTiny) {
            uint32_t w[4] = {};
#pragma unroll
            for (int i = 0; i < V - 1; ++i) {
                if constexpr (ES == 4)
                    w[i] = __builtin_amdgcn_raw_buffer_load_b32(r, (col0 + i) * ES, 0, 0);
                else
                    w[i / 2] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(
                                    r, (col0 + i) * ES, 0, 0)
                                << (16 * (i % 2));
            }
            return (u32x4){w[0], w[1], w[2], w[3]};
        } else {
            return __builtin_amdgcn_raw_buffer_load_b128(r, at(s) * ES, 0, kPolicyStream);
        }
    }
    __device__ __forceinline__ void take(u32x4 w, int s, float* v) const {
        if (EDGE == kPart && s == S - 1) w = shift_down(w, lost * ES);
        E::widen(w, v);
    }
    __device__ __forceinline__ void store(rsrc_t r, int s, const float* v) const {
        const u32x4 w = E::narrow(v);
        if (EDGE == kWhole || s < S - 1 || (EDGE == kPart && !part)) {
            __builtin_amdgcn_raw_buffer_store_b128(w, r, col(s) * ES, 0, kPolicyStore);
            return;
        }
        if (EDGE == kTiny && !part) return;
#pragma unroll
        for (int i = 0; i < V - 1; ++i) {
            if constexpr (ES == 4)
                __builtin_amdgcn_raw_buffer_store_b32(w[i], r, (col(s) + i) * ES, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b16((unsigned short)(w[i / 2] >> (16 * (i % 2))),
                                                      r, (col(s) + i) * ES, 0, 0);
        }
    }

    // V values of a norm weight (32 bits, or the activations' type).
    struct Weight {
        u32x4 w[V == 8 ? 2 : 1];
    };
    // Without a branch on its type or on whether there is one (null: zeros), so
    // that several are on their way together.
    __device__ __forceinline__ Weight load_weight(const char* p, int f32, int s) const {
        Weight k;
        const int es = f32 ? 4 : ES;
        const rsrc_t r = row_rsrc(p, p != nullptr ? cols * es : 0);
        if constexpr (EDGE == kTiny) {
            uint32_t w[8] = {};
#pragma unroll
            for (int i = 0; i < V - 1; ++i) {
                if (es == 4)
                    w[i] = __builtin_amdgcn_raw_buffer_load_b32(r, (col0 + i) * 4, 0, 0);
                else
                    w[i / 2] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(
                                    r, (col0 + i) * 2, 0, 0)
                                << (16 * (i % 2));
            }
            k.w[0] = (u32x4){w[0], w[1], w[2], w[3]};
            if constexpr (V == 8) k.w[1] = (u32x4){w[4], w[5], w[6], w[7]};
        } else {
            k.w[0] = __builtin_amdgcn_raw_buffer_load_b128(r, at(s) * es, 0, kPolicyKeep);
            if constexpr (V == 8)  // past the row for the type of 16 bits
                k.w[1] = __builtin_amdgcn_raw_buffer_load_b128(
                    r, f32 ? at(s) * 4 + 16 : 0x40000000, 0, kPolicyKeep);
        }
        return k;
    }
    __device__ __forceinline__ void take_weight(const Weight& k, int f32, float offset, int s,
                                                float* v) const {
        if (V == 4 || !f32) {
            take(k.w[0], s, v);
        } else {
            uint32_t u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = k.w[i / 4 % (V / 4)][i % 4];
            if (EDGE == kPart && s == S - 1) shift_words(u, lost);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = as_f(u[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] += offset;
    }

    // A packed row: its values and its scale bytes.
    struct KeptRow {
        rsrc_t q, s;
    };
    __device__ __forceinline__ KeptRow kept_row(const Kept& k, int64_t row) const {
        return {row_rsrc(k.q + row * k.q_ld, cols),
                row_rsrc(k.s + row * k.s_ld,
                         (cols + PTORED_CHECKPOINT_BLOCK - 1) / PTORED_CHECKPOINT_BLOCK)};
    }
    __device__ __forceinline__ KeptRaw load_kept(const KeptRow& k, int s) const {
        KeptRaw w;
        w.q = (u32x2){0u, 0u};
        if constexpr (EDGE == kTiny) {
#pragma unroll
            for (int i = 0; i < V - 1; ++i)
                w.q[i / 4] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(k.q, col0 + i, 0, 0)
                              << (8 * (i % 4));
        } else if constexpr (V == 8) {
            w.q = __builtin_amdgcn_raw_buffer_load_b64(k.q, at(s), 0, kPolicyStream);
        } else {
            w.q[0] = __builtin_amdgcn_raw_buffer_load_b32(k.q, at(s), 0, kPolicyStream);
        }
        w.scale = __builtin_amdgcn_raw_buffer_load_b8(k.s, col(s) / PTORED_CHECKPOINT_BLOCK, 0, 0);
        return w;
    }
    // The values kept times `by`; exact products aside, the same as taking them first.
    __device__ __forceinline__ void take_kept(const KeptRaw& w, int s, float by, float* v) const;
    __device__ __forceinline__ void store_kept(const KeptRow& k, int s, const float* v) const;
};

// Threads of a launch as Slots counts on it, with `per` slots each or, where
// a thread's first per - 1 would not all lie inside the row, fewer.
inline int slot_threads(int slots, int& per) {
    for (;; per /= 2) {
        const int threads = ((slots + per - 1) / per + 63) / 64 * 64;
        if (per == 1 || (per - 1) * threads < slots) return threads;
    }
}

// ---------------------------------------------------------------- sums

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t u) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, CTRL, 0xF, 0xF, true);
}
constexpr int kDppXor1 = 0xB1;         // lanes 1 0 3 2 of each quad
constexpr int kDppXor2 = 0x4E;         // lanes 2 3 0 1 of each quad
constexpr int kDppHalfMirror = 0x141;  // lane i of 8 takes 7 - i

// One step of a sum over the wave: adds what CTRL moves into the lanes of the
// rows (of 16 lanes) in ROWS, nothing elsewhere.
template <int CTRL, int ROWS>
__device__ __forceinline__ float add_moved(float x) {
    return x + as_f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_u(x), CTRL, ROWS, 0xF, true));
}
// The wave's sum, in lane 63: inside rows by shifts of 1, 2, 4 and 8 lanes,
// then each row's last lane into the next row, then the half's into the other
// half.  (A shuffle through the LDS per step takes several times as long.)
__device__ __forceinline__ float wave_sum(float x) {
    x = add_moved<0x111, 0xF>(x);
    x = add_moved<0x112, 0xF>(x);
    x = add_moved<0x114, 0xF>(x);
    x = add_moved<0x118, 0xF>(x);
    x = add_moved<0x142, 0xA>(x);
    return add_moved<0x143, 0xC>(x);
}

constexpr int kMaxWaves = 16;  // waves of the largest workgroup

// Sums of K values over the workgroup, in a fixed order.  `red` is one of the
// caller's buffers; the caller alternates between two, so that one barrier
// per sum is enough: a wave writes a buffer again only after the barrier of
// the sum in between, which every wave reaches after it has read this one.
typedef float f32x4 __attribute__((ext_vector_type(4)));
template <int K>
__device__ __forceinline__ void block_sum(f32x4 (*red)[kMaxWaves / 4], float* v) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
    const int waves = (int)blockDim.x >> 6, wave = (int)threadIdx.x >> 6;
    if (waves == 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = as_f((uint32_t)__builtin_amdgcn_readlane((int)as_u(v[k]), 63));
        return;
    }
    if ((threadIdx.x & 63) == 63) {
#pragma unroll
        for (int k = 0; k < K; ++k) red[k][wave / 4][wave % 4] = v[k];
        // the last wave fills its group of four
        for (int w = waves; w % 4 != 0 && wave == waves - 1; ++w)
#pragma unroll
            for (int k = 0; k < K; ++k) red[k][w / 4][w % 4] = 0.0f;
    }
    __syncthreads();
    f32x4 s[K];
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = red[k][0];
    if (waves > 4) {
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] += red[k][1];
    }
    if (waves > 8) {
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] += red[k][2];
    }
    if (waves > 12) {
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] += red[k][3];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = (s[k][0] + s[k][1]) + (s[k][2] + s[k][3]);
}

// ---------------------------------------------------------------- 8 bits

// 2^n for n in [-126, 127]
__device__ __forceinline__ float power_of_2(int n) { return as_f((uint32_t)(n + 127) << 23); }

// Largest magnitude of a block of 32 elements, as bits, in all its lanes: a
// block is 4 lanes of 8 elements or 8 lanes of 4.  The maximum is IEEE 754's,
// which a NaN passes through; bit patterns of non-negative floats compare like
// the values, infinities and NaN above all.
template <int V>
__device__ __forceinline__ uint32_t block_amax(const float* v) {
    float t = __builtin_fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < V; ++i) t = __builtin_elementwise_maximum(t, __builtin_fabsf(v[i]));
    uint32_t m = as_u(t) & 0x7FFFFFFFu;
    m = max(m, dpp<kDppXor1>(m));
    m = max(m, dpp<kDppXor2>(m));
    if constexpr (V == 4) m = max(m, dpp<kDppHalfMirror>(m));
    return m;
}

// A slot's packed form: V bytes and the block's scale byte.  Every lane of the
// wave takes part (slots past the row hold zeros, which do not change its last
// block's largest magnitude).
template <int V>
__device__ __forceinline__ KeptRaw quantise(const float* v) {
    const uint32_t top = block_amax<V>(v);
    const bool finite = top < 0x7F800000u;
    // E: the exponent of amax, one more where amax 2^(6-E) would round to 128
    // (127.5 = 64 * 1.1111111b does, ties to even)
    int e = (int)(top >> 23) - 127 + ((top & 0x7FFFFFu) >= 0x7F0000u ? 1 : 0);
    e = min(max(e, -120), 127);
    // 1.5 2^23 + v 2^(6-E) has the quotient, rounded with ties to even, in its
    // low bits
    const float f = power_of_2(6 - e), m = 12582912.0f;
    KeptRaw k;
    k.q = (u32x2){0u, 0u};
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        uint32_t q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            q[j] = as_u(__builtin_amdgcn_fmed3f(fmaf(v[i + j], f, m), m - 127.0f, m + 127.0f));
        const uint32_t lo = __builtin_amdgcn_perm(q[1], q[0], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(q[3], q[2], 0x04000C0Cu);
        k.q[i / 4] = finite ? lo | hi : 0u;
    }
    k.scale = finite ? (uint32_t)(e + 127) : 255u;
    return k;
}

// The factor 2^(E-6) of a scale byte; NaN for 255.
__device__ __forceinline__ float scale_factor(uint32_t s) {
    // bytes below 7 are never written; they count as 7 rather than leave the
    // exponent's range
    return s == 255u ? as_f(0x7FC00000u) : as_f((max(s, 7u) - 6u) << 23);
}

template <int V>
__device__ __forceinline__ void dequantise(const KeptRaw& k, float by, float* v) {
    const float f = scale_factor(k.scale) * by;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)(int8_t)(k.q[i / 4] >> (8 * (i % 4))) * f;
}

template <int DT, int S, int EDGE>
__device__ __forceinline__ void Slots<DT, S, EDGE>::store_kept(const KeptRow& r, int s,
                                                               const float* v) const {
    const KeptRaw k = quantise<V>(v);
    const int c = col(s);
    if (EDGE == kWhole || s < S - 1 || !part) {
        if constexpr (V == 8)
            __builtin_amdgcn_raw_buffer_store_b64(k.q, r.q, c, 0, kPolicyStore);
        else
            __builtin_amdgcn_raw_buffer_store_b32(k.q[0], r.q, c, 0, kPolicyStore);
    } else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            __builtin_amdgcn_raw_buffer_store_b8((unsigned char)(k.q[i / 4] >> (8 * (i % 4))), r.q,
                                                 c + i, 0, 0);
    }
    if ((c & (PTORED_CHECKPOINT_BLOCK - 1)) == 0)
        __builtin_amdgcn_raw_buffer_store_b8((unsigned char)k.scale, r.s,
                                             c / PTORED_CHECKPOINT_BLOCK, 0, 0);
}

template <int DT, int S, int EDGE>
__device__ __forceinline__ void Slots<DT, S, EDGE>::take_kept(const KeptRaw& w, int s,
                                                              float by, float* v) const {
    KeptRaw k = w;
    if (EDGE == kPart && s == S - 1) {
        const uint64_t u = ((uint64_t)k.q[1] << 32 | k.q[0]) >> (8 * lost);
        k.q = (u32x2){(uint32_t)u, (uint32_t)(u >> 32)};
    }
    dequantise<V>(k, by, v);
}

}  // namespace block
}  // namespace ptored
