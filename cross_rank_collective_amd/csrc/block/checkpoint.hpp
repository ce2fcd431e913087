// checkpoint.hpp -- activations to 8 bits and back.
//
// Bound by memory: 2 or 4 bytes an element on one side, 33/32 on the other.
// Slots are numbered straight through the rows, so that a block of 32 elements
// lies in 4 (or 8) neighbouring lanes (a row takes a whole number of those)
// and narrow rows fill the waves.  A thread takes PER slots and loads all of
// them before it uses the first: 4 (one: 45 us to pack 8192 x 8192 in bf16, 4:
// 34 us), or one where the slots are too few to fill the chip four at a time
// (777 x 1003 in f32: 4.9 against 3.5 us).
#pragma once

#include "block_device.hpp"

namespace ptored {
namespace block {

constexpr int kPackThreads = 256;

// Slot `x` past the row's start, which may be rows further on: `row` and the
// column.  inv = floor(2^32 / row_slots) + 1 where row_slots < 1024: then x <
// 2048 and the quotient is exact.
__device__ __forceinline__ int slot_place(uint32_t x, uint32_t row_slots, uint32_t inv, int64_t& row) {
    const uint32_t q = inv ? __umulhi(x, inv) : x >= row_slots ? 1u : 0u;
    row += q;
    return (int)(x - q * row_slots);
}

// ES bytes each, `n` of them, at p; zeros behind.
template <int ES>
__device__ __forceinline__ u32x4 load_some(const char* p, int n) {
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 16 / ES - 1; ++i) {
        if (i >= n) continue;
        if constexpr (ES == 4)
            w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else if constexpr (ES == 2)
            w[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i % 2));
        else
            w[i / 4] |= (uint32_t) reinterpret_cast<const uint8_t*>(p)[i] << (8 * (i % 4));
    }
    return (u32x4){w[0], w[1], w[2], w[3]};
}

template <int DT, bool TAIL, int PER>
__global__ __launch_bounds__(kPackThreads) void pack_kernel(const PackArgs a, uint32_t row_slots,
                                                            uint32_t inv, int64_t tiles) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t n = tile * (kPackThreads * PER), row0 = n / row_slots;
        const uint32_t x0 = (uint32_t)(n - row0 * row_slots) + threadIdx.x;
        u32x4 w[PER];
        int64_t row[PER];
        int col[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            row[k] = row0;
            col[k] = slot_place(x0 + k * kPackThreads, row_slots, inv, row[k]) * V;
            const char* p = a.x.p + row[k] * a.x.ld + (int64_t)col[k] * E::kBytes;
            w[k] = (u32x4)(0u);
            if (row[k] >= a.rows || col[k] >= a.cols) {
                col[k] = a.cols;  // stores nothing
            } else if (!TAIL || col[k] + V <= a.cols) {
                w[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
            } else {
                w[k] = load_some<E::kBytes>(p, a.cols - col[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            float v[V];
            E::widen(w[k], v);
            const KeptRaw kept = quantise<V>(v);
            if (col[k] >= a.cols) continue;
            int8_t* q = a.k.q + row[k] * a.k.q_ld + col[k];
            if (!TAIL || col[k] + V <= a.cols) {
                if constexpr (V == 8)
                    *reinterpret_cast<u32x2_any*>(q) = kept.q;
                else
                    *reinterpret_cast<u32_any*>(q) = kept.q[0];
            } else {
#pragma unroll
                for (int i = 0; i < V - 1; ++i)
                    if (col[k] + i < a.cols) q[i] = (int8_t)(kept.q[i / 4] >> (8 * (i % 4)));
            }
            if (col[k] % PTORED_CHECKPOINT_BLOCK == 0)
                a.k.s[row[k] * a.k.s_ld + col[k] / PTORED_CHECKPOINT_BLOCK] = (uint8_t)kept.scale;
        }
    }
}

template <int DT, bool TAIL, int PER>
__global__ __launch_bounds__(kPackThreads) void unpack_kernel(const PackArgs a, uint32_t row_slots,
                                                              uint32_t inv, int64_t tiles) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t n = tile * (kPackThreads * PER), row0 = n / row_slots;
        const uint32_t x0 = (uint32_t)(n - row0 * row_slots) + threadIdx.x;
        KeptRaw w[PER];
        int64_t row[PER];
        int col[PER];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            row[k] = row0;
            col[k] = slot_place(x0 + k * kPackThreads, row_slots, inv, row[k]) * V;
            w[k] = KeptRaw{(u32x2){0u, 0u}, 0u};
            if (row[k] >= a.rows || col[k] >= a.cols) {
                col[k] = a.cols;
                continue;
            }
            const int8_t* q = a.k.q + row[k] * a.k.q_ld + col[k];
            w[k].scale = a.k.s[row[k] * a.k.s_ld + col[k] / PTORED_CHECKPOINT_BLOCK];
            if (!TAIL || col[k] + V <= a.cols) {
                if constexpr (V == 8)
                    w[k].q = __builtin_nontemporal_load(reinterpret_cast<const u32x2_any*>(q));
                else
                    w[k].q[0] = __builtin_nontemporal_load(reinterpret_cast<const u32_any*>(q));
            } else {
                const u32x4 u = load_some<1>(reinterpret_cast<const char*>(q), a.cols - col[k]);
                w[k].q = (u32x2){u[0], u[1]};
            }
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (col[k] >= a.cols) continue;
            float v[V];
            dequantise<V>(w[k], 1.0f, v);
            char* p = a.x.p + row[k] * a.x.ld + (int64_t)col[k] * E::kBytes;
            if (!TAIL || col[k] + V <= a.cols) {
                __builtin_nontemporal_store(E::narrow(v), reinterpret_cast<u32x4_any*>(p));
            } else {
#pragma unroll
                for (int i = 0; i < V - 1; ++i)
                    if (col[k] + i < a.cols) E::store1(p + i * E::kBytes, v[i]);
            }
        }
    }
}

template <int DT, bool PACK, int PER>
static int launch_pack(const PackArgs& a, uint32_t row_slots, int64_t slots, hipStream_t stream) {
    constexpr uint32_t kTile = kPackThreads * PER;
    const bool tail = a.cols % Elem<DT>::V != 0;
    uint32_t inv = row_slots < 1024 ? (uint32_t)((uint64_t(1) << 32) / row_slots + 1) : 0;
    int64_t tiles = (slots + kTile - 1) / kTile;
    const void* k =
        PACK ? (tail ? reinterpret_cast<const void*>(pack_kernel<DT, true, PER>)
                     : reinterpret_cast<const void*>(pack_kernel<DT, false, PER>))
             : (tail ? reinterpret_cast<const void*>(unpack_kernel<DT, true, PER>)
                     : reinterpret_cast<const void*>(unpack_kernel<DT, false, PER>));
    const int64_t grid = tiles < (1 << 22) ? tiles : 1 << 22;
    void* args[] = {const_cast<PackArgs*>(&a), &row_slots, &inv, &tiles};
    return hipLaunchKernel(k, dim3((uint32_t)grid), dim3(kPackThreads), args, 0, stream) ==
                   hipSuccess
               ? kOk
               : kFailed;
}

template <int DT, bool PACK>
int pack_launch(const PackArgs& a, hipStream_t stream) {
    const uint32_t row_slots = (uint32_t)(((int64_t)a.cols + 31) / 32 * 32 / Elem<DT>::V);
    const int64_t slots = a.rows * (int64_t)row_slots;
    return slots >= 1 << 20 ? launch_pack<DT, PACK, 4>(a, row_slots, slots, stream)
                            : launch_pack<DT, PACK, 1>(a, row_slots, slots, stream);
}

}  // namespace block
}  // namespace ptored
