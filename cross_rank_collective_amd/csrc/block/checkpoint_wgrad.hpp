// checkpoint_wgrad.hpp -- a projection's weight gradient from its packed input.
//
//     dw[o, i] = sum_t dy[t, o] x[t, i],   x[t, i] = q 2^(E-6)
//
// A matrix product over the tokens, both operands with the sum's index as the
// slow one.  The values kept are exact in bfloat16, so x enters the matrix
// instructions without loss; so does dy, as one bfloat16 (bf16) or the exact
// sum of three (f32, but for what lies below bfloat16's smallest step, 2^-133):
// products are exact and sums in binary32.  For f16, dy is used as it is and x
// in f16, which holds a block exactly if its exponent is in [-18, 15]; a
// workgroup that meets another block (or a NaN) starts again with dy as the
// exact sum of two bfloat16.
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
//
// What it took, on one MI355X (bf16): 8192 tokens x 4096 x 4096 in tiles of 256
// x 256 250 us, 1.1 PFLOP/s (a plain matrix product of the same layout by the
// vendor's library 286 us from bfloat16 operands; 213 us at the rate of its
// 8192^3 product).  The matrix cores are busy 53% of the cycles, and the card
// lowers its clock to 1.95 GHz; the LDS is busy 40%.  Staging x takes 44
// vector instructions for each 16 values, which a larger tile shares among more
// products: 128 x 128 tiles reach 0.65 PFLOP/s.  Those have two groups of
// waves, each for half of the tokens, joined in the LDS at the end: 1024 x 2048
// x 2048 20 us, with one group 25 us.
#pragma once

#include <type_traits>

#include "block_device.hpp"

namespace ptored {
namespace block {

constexpr int kStep = 32;  // tokens staged at a time for each group of waves

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

// HALF: the operands are f16.
template <int DT, bool HALF>
constexpr int planes_of() {
    return DT == PTORED_BF16 || HALF ? 1 : DT == PTORED_F16 ? 2 : 3;
}

// 8 elements of dy as words: as loaded, split into bfloat16 planes on the way
// to the LDS.
template <int DT>
struct DyChunk {
    u32x4 w[DT == PTORED_F32 ? 2 : 1];
};

// An edge chunk's elements from where they were loaded to their places, `n`
// bytes on.
template <int DT>
__device__ __forceinline__ void move_up(DyChunk<DT>& c, int n) {
    if constexpr (DT == PTORED_F32) {  // whole words, over 32 bytes
#pragma unroll
        for (int b = 16; b >= 4; b /= 2) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t far = i + b / 4 < 8 ? c.w[(i + b / 4) / 4 % 2][(i + b / 4) % 4] : 0u;
                w[i] = n & b ? far : c.w[i / 4][i % 4];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) c.w[i / 4][i % 4] = w[i];
        }
    } else {
        c.w[0] = shift_down(c.w[0], n);
    }
}

// The `n` elements of ES bytes at `p`, fewer than a chunk has, zeros behind.
template <int ES>
__device__ __forceinline__ void load_few(const char* p, int n, u32x4* w) {
    constexpr int kCount = ES == 1 ? 16 : 8;
    uint32_t u[kCount * ES / 4] = {};
#pragma unroll
    for (int i = 0; i < kCount - 1; ++i) {
        if (i >= n) continue;
        if constexpr (ES == 4)
            u[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else if constexpr (ES == 2)
            u[i / 2] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i % 2));
        else
            u[i / 4] |= (uint32_t) reinterpret_cast<const uint8_t*>(p)[i] << (8 * (i % 4));
    }
#pragma unroll
    for (int i = 0; i < kCount * ES / 4; ++i) w[i / 4][i % 4] = u[i];
}

// Upper halves of two words, lo's first.
__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi) {
    return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// Plane 0 is the value's upper half (truncated, so that it cannot overflow),
// each next plane that of the exact remainder; infinities and NaN are in
// plane 0 alone.
template <int DT, bool HALF>
__device__ __forceinline__ void split_dy(const DyChunk<DT>& c, u32x4* plane) {
    if constexpr (DT == PTORED_BF16 || HALF) {
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
        for (int k = 0; k < planes_of<DT, HALF>(); ++k) {
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

// 16 packed values of one block and its scale byte.
struct KeptChunk {
    u32x4 w;
    uint32_t scale;
};

// The chunk's values as bfloat16 (exact: at most 8 significant bits), or f16.
template <bool HALF>
__device__ __forceinline__ void widen_kept(const KeptChunk& c, u32x4* out) {
    const float f = scale_factor(c.scale);
    uint32_t v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = as_u((float)(int8_t)(c.w[i / 4] >> (8 * (i % 4))) * f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (HALF)
            out[i / 4][i % 4] = __builtin_bit_cast(
                uint32_t, __builtin_amdgcn_cvt_pkrtz(as_f(v[2 * i]), as_f(v[2 * i + 1])));
        else
            out[i / 4][i % 4] = upper_halves(v[2 * i], v[2 * i + 1]);
    }
}

// Whether f16 does not hold the chunk: an exponent outside [-18, 15] (q
// 2^(E-6) would leave the grid of 2^-24 or pass 65504) with values, or a NaN.
__device__ __forceinline__ bool leaves_half(const KeptChunk& c) {
    const bool out = c.scale - 109u > 33u;
    return out && (c.scale == 255u || (c.w[0] | c.w[1] | c.w[2] | c.w[3]) != 0);
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

// Rows of dy or of x that do not end with a whole chunk (8 and 16 elements).
enum : int {
    kWholeChunks = 0,
    kPartChunks = 1,  // the last chunk is loaded so that it ends with the row, and moved
    kFewElements = 2  // a row shorter than a chunk: element by element
};

// A tile's sums over tokens [begin, end), from column m0 of dy and n0 of x, by
// KG groups of waves WM x WN, each wave computing TM x TN blocks of 32 x 32
// over its group's share of the tokens.  Returns whether a chunk of x was not
// held by HALF's operands.
template <int DT, bool HALF, int WM, int WN, int KG, int TM, int TN, int EDGE>
__device__ __forceinline__ bool wgrad_tile(const WgradArgs& a, char* lds, int m0, int n0,
                                           int64_t begin, int64_t end, f32x16 (&acc)[TM][TN]) {
    constexpr int STEP = kStep * KG;
    constexpr int kThreads = WM * WN * KG * 64;
    constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
    constexpr int P = planes_of<DT, HALF>();
    constexpr int kRowA = BM * 2, kRowB = BN * 2;
    constexpr int kBytesA = STEP * kRowA, kBytesB = STEP * kRowB;
    constexpr int kBytes = P * kBytesA + kBytesB;
    constexpr int kChunksA = STEP * BM / 8 / kThreads, kChunksB = STEP * BN / 16 / kThreads;
    constexpr int kRowsA = kThreads / (BM / 8), kRowsB = kThreads / (BN / 16);
    static_assert(kChunksA * kRowsA == STEP && kChunksB * kRowsB == STEP,
                  "whole chunks per thread");
    static_assert(kRowsA % 4 == 0 && kRowsB % 4 == 0, "a thread's rows share their swizzle");
    const int tid = (int)threadIdx.x;
    const int wave = (tid >> 6) % (WM * WN), group = (tid >> 6) / (WM * WN);
    // an even number: the loop takes two
    const int steps = 2 * (int)((end - begin + 2 * STEP - 1) / (2 * STEP));
    bool left_half = false;

    // This thread's chunks of a step: rows tA + c kRowsA of dy, tB + c kRowsB
    // of x.  A chunk that would pass the end of a row is loaded from the row's
    // last whole chunk instead: what lies past the end is not stored, and with
    // EDGE the elements before it are moved to their places (shA, shB).
    using E = Elem<DT>;
    const int tA = tid / (BM / 8), colA = m0 + tid % (BM / 8) * 8;
    const int tB = tid / (BN / 16), colB = n0 + tid % (BN / 16) * 16;
    const int fromA = min(colA, max(a.outs - 8, 0)), fromB = min(colB, max(a.cols - 16, 0));
    const char* pa = a.dy + (begin + tA) * a.dy_ld + (int64_t)fromA * E::kBytes;
    const int8_t* pq = a.x.q + (begin + tB) * a.x.q_ld + fromB;
    const uint8_t* ps =
        a.x.s + (begin + tB) * a.x.s_ld + min(colB, a.cols - 1) / PTORED_CHECKPOINT_BLOCK;
    const int shA = min(colA - fromA, 7) * E::kBytes, shB = min(colB - fromB, 15);

    struct Tokens {
        DyChunk<DT> dy[kChunksA];
        KeptChunk kept[kChunksB];
    };
    Tokens set0, set1;
    // Loads the next tokens, STEP of them unless FIRST.
    int64_t rowsA = kRowsA * a.dy_ld, rowsQ = kRowsB * a.x.q_ld, rowsS = kRowsB * a.x.s_ld;
    auto fetch = [&](auto first, Tokens& set, int tokens) {
        constexpr bool FIRST = decltype(first)::value;
#pragma unroll
        for (int c = 0; c < kChunksA; ++c) {
            const char* p = pa + c * rowsA;
            set.dy[c] = DyChunk<DT>{};
            if (FIRST && tA + c * kRowsA >= tokens) continue;
            if (EDGE == kFewElements && a.outs < 8) {
                load_few<E::kBytes>(p, a.outs, set.dy[c].w);
            } else {
                set.dy[c].w[0] = *reinterpret_cast<const u32x4_any*>(p);
                if constexpr (DT == PTORED_F32)
                    set.dy[c].w[1] = *reinterpret_cast<const u32x4_any*>(p + 16);
            }
        }
#pragma unroll
        for (int c = 0; c < kChunksB; ++c) {
            set.kept[c] = KeptChunk{(u32x4)(0u), 127u};
            if (FIRST && tB + c * kRowsB >= tokens) continue;
            const int8_t* q = pq + c * rowsQ;
            if (EDGE == kFewElements && a.cols < 16)
                load_few<1>(reinterpret_cast<const char*>(q), a.cols, &set.kept[c].w);
            else
                set.kept[c].w = *reinterpret_cast<const u32x4_any*>(q);
            set.kept[c].scale = ps[c * rowsS];
        }
    };
    auto advance = [&](int64_t tokens) {
        pa += tokens * a.dy_ld;
        pq += tokens * a.x.q_ld;
        ps += tokens * a.x.s_ld;
    };
    const int atA = lds_chunk(tA, tid % (BM / 8), kRowA);
    const int atB0 = lds_chunk(tB, tid % (BN / 16) * 2, kRowB);
    const int atB1 = lds_chunk(tB, tid % (BN / 16) * 2 + 1, kRowB);
    auto stage_a = [&](Tokens& set, char* buf, int c) {
        u32x4 plane[P];
        if constexpr (EDGE != kWholeChunks) move_up<DT>(set.dy[c], shA);
        split_dy<DT, HALF>(set.dy[c], plane);
#pragma unroll
        for (int p = 0; p < P; ++p)
            *reinterpret_cast<u32x4*>(buf + p * kBytesA + c * kRowsA * kRowA + atA) = plane[p];
    };
    auto stage_b = [&](Tokens& set, char* buf, int c) {
        u32x4 v[2];
        // keeps the unpacking here: right after the loads it would wait for them
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t u = set.kept[c].w[i];
            asm volatile("" : "+v"(u));
            set.kept[c].w[i] = u;
        }
        asm volatile("" : "+v"(set.kept[c].scale));
        if constexpr (EDGE != kWholeChunks) set.kept[c].w = shift_down(set.kept[c].w, shB);
        if constexpr (HALF) left_half |= leaves_half(set.kept[c]);
        widen_kept<HALF>(set.kept[c], v);
        char* at = buf + P * kBytesA + c * kRowsB * kRowB;
        *reinterpret_cast<u32x4*>(at + atB0) = v[0];
        *reinterpret_cast<u32x4*>(at + atB1) = v[1];
    };
    auto stage = [&](Tokens& set, char* buf) {
#pragma unroll
        for (int c = 0; c < kChunksB; ++c) stage_b(set, buf, c);
#pragma unroll
        for (int c = 0; c < kChunksA; ++c) stage_a(set, buf, c);
    };

#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = (f32x16)(0.0f);
    const int pm = wave / WN * TM, pn = wave % WN * TN;  // the wave's 64-byte pieces

    struct Fragments {
        b8 a[P][TM], b[TN];
    };
    auto read = [&](const char* buf, int k, Fragments& f) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
            f.b[j] = read_fragment(buf + P * kBytesA, (group * 2 + k) * 16, pn + j, kRowB);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < TM; ++i)
                f.a[p][i] = read_fragment(buf + p * kBytesA, (group * 2 + k) * 16, pm + i, kRowA);
    };
    auto multiply = [&](const Fragments& f) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    if constexpr (HALF)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                            __builtin_bit_cast(h8, f.a[p][i]), __builtin_bit_cast(h8, f.b[j]),
                            acc[i][j], 0, 0, 0);
                    else
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[p][i], f.b[j],
                                                                           acc[i][j], 0, 0, 0);
                }
    };

    // The pipeline, in steps of 32 tokens a group: loaded into registers four
    // steps ahead, staged in the LDS two steps ahead, read as fragments 16
    // tokens ahead.  One barrier a step, between its halves: behind it the next
    // step's buffer, staged in the last step, is whole, and the one that this
    // step stages into has been read.  Staging belongs to the second half, so
    // that its writes have landed when the next barrier waits for them (with
    // the first half's: 7% slower).  (Past the last step stale registers are
    // staged and read; nothing uses them.)
    using Yes = std::integral_constant<bool, true>;
    using No = std::integral_constant<bool, false>;
    Fragments even, odd;
    char *b0 = lds, *b1 = lds + kBytes, *b2 = lds + 2 * kBytes;
    // The order of a half's instructions: the fragments' reads between the
    // first products, the arithmetic of the staging spread over the others.
    auto order = [] {
#pragma unroll
        for (int i = 0; i < P * TM * TN; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // matrix instruction
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // LDS reads
            __builtin_amdgcn_sched_group_barrier(0x002, 14, 0);  // vector arithmetic
        }
    };
    auto step = [&](Tokens& set, bool more) {
        __builtin_amdgcn_sched_barrier(0);
        read(b0, 1, odd);
        multiply(even);
        order();
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        read(b1, 0, even);
        multiply(odd);
        stage(set, b2);
        fetch(No{}, set, STEP);
        pa += more ? a.dy_ld * STEP : 0;
        pq += more ? a.x.q_ld * STEP : 0;
        ps += more ? a.x.s_ld * STEP : 0;
        order();
        __builtin_amdgcn_sched_barrier(0);
        char* t = b0;
        b0 = b1;
        b1 = b2;
        b2 = t;
    };
    // The first two steps take what does not fill two whole ones (perhaps only
    // the second does anything).
    const int some = (int)(end - begin - (int64_t)(steps - 2) * STEP);  // 1 to 2 STEP
    const int first = some > STEP ? some - STEP : 0;
    fetch(Yes{}, set0, first);
    advance(first);
    fetch(Yes{}, set1, some - first);
    stage(set0, b0);
    stage(set1, b1);
    if (steps > 2) {
        advance(some - first);
    } else {  // nothing is left to load; what the loop loads is the first row, unused
        advance(-first);
        pa -= tA * a.dy_ld;
        pq -= tB * a.x.q_ld;
        ps -= tB * a.x.s_ld;
        rowsA = rowsQ = rowsS = 0;
    }
    fetch(No{}, set0, STEP);
    advance(steps > 3 ? STEP : 0);
    fetch(No{}, set1, STEP);
    advance(steps > 4 ? STEP : 0);
#pragma unroll
    for (int c = 0; c < kChunksB; ++c) {  // in registers as words, not as bytes to widen at the loop's top
        asm volatile("" : "+v"(set0.kept[c].scale));
        asm volatile("" : "+v"(set1.kept[c].scale));
    }
    __syncthreads();
    read(b0, 0, even);
    for (int s = 0; s < steps; s += 2) {
        step(set0, s + 5 < steps);
        step(set1, s + 6 < steps);
    }
    return left_half;
}

template <int DT, int WM, int WN, int KG, int TM, int TN, int EDGE>
__global__ __launch_bounds__(WM* WN* KG * 64) void wgrad_kernel(const WgradArgs a) {
    constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
    __shared__ __attribute__((aligned(128))) char
        lds[3 * kStep * KG * 2 * (planes_of<DT, false>() * BM + BN)];
    __shared__ int left_half;

    const int lane = (int)threadIdx.x & 63;
    const int wave = (int)(threadIdx.x >> 6) % (WM * WN), group = (int)(threadIdx.x >> 6) / (WM * WN);
    // Workgroups go to the 8 dies in turn: each die gets consecutive tiles of
    // the order in which 4 rows of tiles advance together, so that its cache
    // serves most reads of both operands.
    const int tiles = a.tiles_m * a.tiles_n;
    const int total = tiles * a.splits;
    int id = (int)blockIdx.x;
    {
        const int die = id % 8, each = total / 8, rest = total % 8;
        id = die * each + (die < rest ? die : rest) + id / 8;
    }
    const int split = id / tiles, in_split = id % tiles;
    const int band = in_split / (4 * a.tiles_n), band_rows = min(4, a.tiles_m - band * 4);
    const int in_band = in_split - band * 4 * a.tiles_n;
    const int m0 = (band * 4 + in_band % band_rows) * BM, n0 = in_band / band_rows * BN;
    const int64_t begin = split * a.rows_per_split;
    const int64_t end = begin + a.rows_per_split < a.rows ? begin + a.rows_per_split : a.rows;

    f32x16 acc[TM][TN];
    if constexpr (DT == PTORED_F16) {
        const bool left =
            wgrad_tile<DT, true, WM, WN, KG, TM, TN, EDGE>(a, lds, m0, n0, begin, end, acc);
        if (threadIdx.x == 0) left_half = 0;
        __syncthreads();
        if (left) left_half = 1;
        __syncthreads();
        if (left_half)
            wgrad_tile<DT, false, WM, WN, KG, TM, TN, EDGE>(a, lds, m0, n0, begin, end, acc);
    } else {
        wgrad_tile<DT, false, WM, WN, KG, TM, TN, EDGE>(a, lds, m0, n0, begin, end, acc);
    }

    const int pm = wave / WN * TM, pn = wave % WN * TN;
    if constexpr (KG == 2) {
        // each group takes half of the blocks and leaves the other half's sums
        // to the other group
        static_assert(TM % 2 == 0, "halves");
        float* mine = reinterpret_cast<float*>(lds) + (group * WM * WN + wave) * (TM / 2 * TN * 1024);
        float* other =
            reinterpret_cast<float*>(lds) + ((1 - group) * WM * WN + wave) * (TM / 2 * TN * 1024);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TM / 2; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    other[((i * TN + j) * 16 + r) * 64 + lane] =
                        group ? acc[i][j][r] : acc[TM / 2 + i][j][r];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TM / 2; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float v = mine[((i * TN + j) * 16 + r) * 64 + lane];
                    // the lower tokens first, in both groups
                    acc[i][j][r] = group ? v + acc[TM / 2 + i][j][r] : acc[i][j][r] + v;
                }
    }

    // Register r of a 32 x 32 block is row 8 (r / 4) + 4 (lane / 32) + r % 4,
    // column lane % 32.
#pragma unroll
    for (int i = 0; i < TM / KG; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int col = n0 + (pn + j) * 32 + (lane & 31);
            if (col >= a.cols) continue;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = m0 + (pm + group * (TM / KG) + i) * 32 + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
                if (row >= a.outs) continue;
                float v = acc[i][j][r];
                if (a.splits > 1) {
                    a.ws[((int64_t)split * a.outs + row) * a.ws_ld + col] = v;
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

// dw (+)= the splits' sums.  A workgroup takes 64 times 4 columns of a row, 4
// threads each for every fourth split, joined in the LDS in a fixed order.
constexpr int kJoinLanes = 64, kJoinGroups = 4;
template <int DT>
__global__ __launch_bounds__(kJoinLanes* kJoinGroups) void wgrad_join_kernel(const WgradArgs a) {
    __shared__ f32x4 part[kJoinGroups][kJoinLanes];
    const int lane = (int)threadIdx.x % kJoinLanes, group = (int)threadIdx.x / kJoinLanes;
    const int col = ((int)blockIdx.x * kJoinLanes + lane) * 4;
    const int64_t step = (int64_t)a.outs * a.ws_ld;
    for (int row = (int)blockIdx.y; row < a.outs; row += (int)gridDim.y) {
        f32x4 sum = (f32x4)(0.0f);
        if (col < a.cols) {
            const float* ws = a.ws + (int64_t)row * a.ws_ld + col;
#pragma unroll 4
            for (int s = group; s < a.splits; s += kJoinGroups)
                sum += *reinterpret_cast<const f32x4*>(ws + s * step);
        }
        part[group][lane] = sum;
        __syncthreads();
        if (group == 0 && col < a.cols) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = (part[0][lane][i] + part[1][lane][i]) + (part[2][lane][i] + part[3][lane][i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (col + i >= a.cols) continue;
                if (a.dw_f32) {
                    float* p = reinterpret_cast<float*>(a.dw + row * a.dw_ld) + col + i;
                    *p = a.accumulate ? *p + v[i] : v[i];
                } else {
                    char* p = a.dw + row * a.dw_ld + (int64_t)(col + i) * Elem<DT>::kBytes;
                    if (a.accumulate) v[i] += Elem<DT>::load1(p);
                    Elem<DT>::store1(p, v[i]);
                }
            }
        }
        __syncthreads();
    }
}

template <int DT, int WM, int WN, int KG, int TM, int TN>
static const void* wgrad_pick(const WgradArgs& a, int& threads) {
    threads = WM * WN * KG * 64;
    if (a.outs % 8 != 0 || a.cols % 16 != 0)
        return reinterpret_cast<const void*>(wgrad_kernel<DT, WM, WN, KG, TM, TN, kPartChunks>);
    return reinterpret_cast<const void*>(wgrad_kernel<DT, WM, WN, KG, TM, TN, kWholeChunks>);
}

template <int DT>
int wgrad_launch(const WgradArgs& a, hipStream_t stream) {
    void* args[] = {const_cast<WgradArgs*>(&a)};
    if (a.splits > 0) {
        const dim3 grid((uint32_t)(a.tiles_m * a.tiles_n) * (uint32_t)a.splits);
        int threads = 256;
        const void* k;
        if (a.shape == kWgradFew) {
            k = reinterpret_cast<const void*>(wgrad_kernel<DT, 2, 2, 1, 2, 2, kFewElements>);
        } else if constexpr (DT == PTORED_F32) {
            k = wgrad_pick<DT, 2, 4, 1, 2, 2>(a, threads);  // 128 x 256
        } else {
            k = a.shape == kWgradWide ? wgrad_pick<DT, 2, 4, 1, 4, 2>(a, threads)
                                      : wgrad_pick<DT, 2, 2, 2, 2, 2>(a, threads);
        }
        if (hipLaunchKernel(k, grid, dim3((uint32_t)threads), args, 0, stream) != hipSuccess)
            return kFailed;
    }
    if (a.splits == 1) return kOk;
    const dim3 grid((uint32_t)((a.cols + 4 * kJoinLanes - 1) / (4 * kJoinLanes)),
                    (uint32_t)(a.outs < 32768 ? a.outs : 32768));
    return hipLaunchKernel(reinterpret_cast<const void*>(wgrad_join_kernel<DT>), grid,
                           dim3(kJoinLanes * kJoinGroups), args, 0, stream) == hipSuccess
               ? kOk
               : kFailed;
}

}  // namespace block
}  // namespace ptored
