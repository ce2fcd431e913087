// product.hpp -- the matrix products of the gated feed-forward block.
//
//     kForward  g = x Wg^T, u = x Wu^T, y = f(g) u     sums over columns
//     kInput    dx = dg Wg + du Wu                     over features, both pairs in turn
//     kWeight   dWg = dg^T x, dWu = du^T x             over tokens
//
// An operand's sum index lies along its rows (kAlong) or across them (kAcross);
// either way it is staged in the LDS as it comes from memory, kStepBytes of
// each row along k (64 elements of 16 bits, 32 of 32) and as many rows across.
// What differs is how fragments are read: along rows a lane's 16 bytes at once,
// across them by transposing loads (16 bits: 16 lanes fetch 4 rows x 16
// columns and receive 4 rows of one column each) or word by word (32 bits).
// A lane's fragment is 16 bytes along k of one row of the product: elements
// 0-7 of 16 for lanes 0-31 and 8-15 for the others (0-3 of 8 and 4-7 in 32
// bits), in both layouts alike, so that any two operands match.
//
// The LDS is a ring of NS buffers.  While a workgroup multiplies out of one, the
// loads of the next steps are on their way to the others.  One barrier a step,
// before its last quarter, whose fragments are then in registers: behind it the
// next step's buffer is whole and this step's is free, so the next loads are
// asked for at once and the next step's first fragments are read under the last
// quarter's products.
//
// kDirect loads go straight to the LDS (16 bytes a lane); they need rows that
// start at multiples of 16 bytes and hold whole chunks.  Other matrices go
// through registers (kHeld), a chunk that would pass the end of a row loaded from
// the row's last whole chunk and moved.  kSplit (F32) stores each value as three
// bfloat16 on the way and multiplies six pairs of them: at 16 times the rate of
// the matrix instructions for F32, 2.7 times fewer of their cycles.
//
// Large products are bound by the matrix cores, at the clock that the card's power
// leaves them: 62% busy at 1.7 GHz, bank conflicts 1% of the forward pass's cycles,
// where its blocks are turned, and none of the gradients'.  bf16, us (and the vendor's
// library's product of the same sizes, without activations): forward, 4096 tokens,
// 4096 columns, 2 x 12288 features 593-640, 1.29-1.39 PFLOP/s (631), 2 x 4096 217
// (172); 8192 tokens, 4096 columns, 8192 features: input's gradient 880 (891), the
// weights' 880 (1012).  Measured and not taken: four waves of 128 x 128 (829 TFLOP/s where
// eight of 128 x 64 reach 1100), steps of 64 bytes in rings of 4 or 5, waves'
// priorities (slower, both), a load between any two products (no gain).
// F32, gradients of 1024 tokens, 1536 columns, 4096 features: 461 us with F32's
// own instructions, 328-340 split.
#pragma once

#include <type_traits>

#include "few.hpp"

namespace ptored {
namespace step {

using namespace block;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr uint32_t kNowhere = 0x80000010u;  // past every buffer resource, 16 bytes before it too: reads as zeros

// Address of LDS memory as the hardware takes it.
__device__ __forceinline__ uint32_t lds_address(const char* p) {
    return (uint32_t)(uintptr_t)(lds_char*)p;
}

// 16 bytes a lane from `off` + `more` behind the resource's base to the LDS at `to`
// (the same for all lanes, as `more` is) + 16 x lane.  The compiler does not see the write:
// barriers with a wait order it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is reserved, so every user sets it first
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t off, uint32_t more, uint32_t to) {
    asm volatile(
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, %3 offen lds"
        :
        : "v"(off), "s"(rsrc), "s"(to), "s"(more)
        : "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ u32x4 rsrc_words(const char* base) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return (u32x4){(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p),
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(p >> 32) & 0xFFFFu)),
                   0x7FFFFFFFu, 0x00020000u};
}

// Where rows of STEP bytes keep a chunk: any 8 rows that begin at a multiple of 8,
// and any 16 at one of 16, keep the same chunk in different banks.
template <int STEP>
__device__ __forceinline__ int swizzle(int row) {
    return (STEP == 128 ? row & 7 : row >> 1 & 3) ^ (row >> 3 & 1);
}

// A tile's share of one operand: EXT rows of the product, STEP bytes along k.
// HALVES: the tile's upper half are a second matrix's rows of the same numbers.
template <int DT, int LAYOUT, int EXT, int STEP, int THREADS, bool DIRECT, bool HALVES>
struct Side {
    using E = Elem<DT>;
    static constexpr int ES = E::kBytes, V = 16 / ES;
    static constexpr int kDepth = STEP / ES;  // k's a step
    static constexpr int kRow = LAYOUT == kAlong ? STEP : EXT * ES;
    static constexpr int kBytes = EXT * STEP;
    static constexpr int kPerRow = kRow / 16;
    static constexpr int kLoads = kBytes / 16 / THREADS;
    static constexpr int kRows = THREADS / kPerRow;  // LDS rows that one load of all threads covers
    static_assert(kRows % (LAYOUT == kAlong ? 16 : 4) == 0, "a thread's rows share their swizzle");
    // Chunks that end with a row are loaded from up to a chunk before their place.
    static constexpr int kBack = DIRECT ? 0 : 16;
    static_assert(LAYOUT == kAlong || EXT * 2 >= 256, "four pieces of 64 bytes to permute");
    static_assert(!HALVES || (LAYOUT == kAlong && kLoads % 2 == 0), "halves are whole loads");

    // bytes from the operand's place, or kNowhere; kAcross: of the first chunk, the
    // next ones `pitch` on
    uint32_t off[LAYOUT == kAlong ? kLoads : 1];
    uint32_t pitch;
    int depth;             // kAlong: k of this thread's chunks in a step; kAcross: its first row's
    int moved;             // kAcross: elements from where the chunks are loaded to where they belong
    bool edge;             // some lane of the wave has moved chunks

    // A step's chunks in registers.
    struct Held {
        u32x4 w[kLoads];
        int by;    // kAlong: elements from where the chunks were loaded to where they belong
        bool cut;  // some lane has such
    };

    // The thread's chunks of the product's rows [first, first + EXT) of `total`.
    // `up_ld`: the pitch of the second matrix.
    __device__ __forceinline__ void init(int64_t first, int64_t total, int64_t ld, int64_t up_ld) {
        const int pos = (int)threadIdx.x % kPerRow, row0 = (int)threadIdx.x / kPerRow;
        moved = 0;
        if constexpr (LAYOUT == kAlong) {
            const int c = pos ^ swizzle<STEP>(row0);
            depth = c * V;
#pragma unroll
            for (int q = 0; q < kLoads; ++q) {
                const int row = row0 + (HALVES ? q % (kLoads / 2) : q) * kRows;
                off[q] = first + row < total ? (uint32_t)(row * (second(q) ? up_ld : ld)) + c * 16 + kBack
                                             : kNowhere;
            }
        } else {
            const int c = ((pos >> 2 ^ (row0 & 3)) << 2) | (pos & 3);
            depth = row0;
            int64_t col = first + c * V;
            const bool in = col < total;
            if (!DIRECT && in && col + V > total) {
                const int64_t from = total > V ? total - V : 0;
                moved = (int)(col - from);
                col = from;
            }
            // (the base lies kBack before the tile's first column, for moved ones)
            off[0] = in ? (uint32_t)(row0 * ld + (col - first) * ES + kBack) : kNowhere;
            pitch = (uint32_t)(kRows * ld);
        }
        edge = __ballot(moved != 0) != 0;
    }

    // Where chunk q of a step is loaded from; `left` k's remain, fewer than a step
    // takes only in a row's last one.
    template <bool LAST>
    __device__ __forceinline__ uint32_t place(int q, int left) const {
        const uint32_t at = off[LAYOUT == kAlong ? q : 0];
        if (!LAST) return at;
        return (LAYOUT == kAlong ? depth : depth + q * kRows) >= left ? kNowhere : at;
    }
    __device__ __forceinline__ uint32_t more(int q) const { return LAYOUT == kAlong ? 0u : q * pitch; }
    static __device__ __forceinline__ bool second(int q) { return HALVES && q >= kLoads / 2; }

    __device__ __forceinline__ void load_direct(const char* p, const char* p2, int left, uint32_t to) const {
        const u32x4 r = rsrc_words(p), r2 = HALVES ? rsrc_words(p2) : r;
        const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        auto each = [&](auto last) {
#pragma unroll
            for (int q = 0; q < kLoads; ++q)
                load_to_lds(second(q) ? r2 : r, place<decltype(last)::value>(q, left), more(q),
                            to + q * (THREADS * 16) + wave * 1024);
        };
        if (left >= kDepth)
            each(std::false_type{});
        else
            each(std::true_type{});
    }

    // The same to registers, without a branch: after one, every wait for a load
    // would be one for all that are younger too (501 x 1003 x 2501 f16 27.5 us).
    // SHORT: one operand's rows, of `extent` elements, do not hold a chunk; both come
    // element by element.
    template <bool SHORT>
    __device__ __forceinline__ void load_held(Held& h, const char* p, const char* p2, int left,
                                              int64_t extent) const {
        const rsrc_t r = row_rsrc(p - kBack, 0x7FFFFFFF), r2 = HALVES ? row_rsrc(p2 - kBack, 0x7FFFFFFF) : r;
        if constexpr (!SHORT) {
            // of a chunk that the row's end cuts, what ends with the row
            h.by = LAYOUT == kAlong && depth < left ? max(depth + V - left, 0) : 0;
            h.cut = LAYOUT == kAlong && left < kDepth;
#pragma unroll
            for (int q = 0; q < kLoads; ++q) {
                const uint32_t at = off[LAYOUT == kAlong ? q : 0] - h.by * ES;
                h.w[q] = __builtin_amdgcn_raw_buffer_load_b128(
                    second(q) ? r2 : r,
                    (int)((LAYOUT == kAlong ? depth : depth + q * kRows) < left ? at : kNowhere), (int)more(q), 0);
            }
        } else {
            h.by = 0;
            h.cut = false;
            const int64_t inside = LAYOUT == kAlong ? left - depth : extent;
#pragma unroll
            for (int q = 0; q < kLoads; ++q) {
                const uint32_t from = place<true>(q, left);
                uint32_t w[4] = {};
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int at = (int)(i < inside && from != kNowhere ? from + i * ES : kNowhere);
                    if constexpr (ES == 4)
                        w[i] = __builtin_amdgcn_raw_buffer_load_b32(second(q) ? r2 : r, at, (int)more(q), 0);
                    else
                        w[i / 2] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(second(q) ? r2 : r, at,
                                                                                   (int)more(q), 0)
                                    << (16 * (i % 2));
                }
                h.w[q] = (u32x4){w[0], w[1], w[2], w[3]};
            }
        }
    }
    // F32 as the exact sum of three bfloat16, each a tile of its own: the value's
    // upper half (truncated, so that it cannot overflow), that of the exact
    // remainder, and what is left of it.
    static constexpr int kPlane = EXT * STEP / 2;
    __device__ __forceinline__ void store_split(const Held& h, char* to) const {
        const int row0 = (int)threadIdx.x / kPerRow, pos = (int)threadIdx.x % kPerRow;
        const bool any = LAYOUT == kAlong ? h.cut : edge;
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
            const int row = row0 + q * kRows;
            u32x4 w = h.w[q];
            if (__builtin_expect(any, 0)) w = shift_down(w, (LAYOUT == kAlong ? h.by : moved) * ES);
            int at;
            if constexpr (LAYOUT == kAlong) {  // rows of STEP / 2 bytes
                const int c = pos ^ swizzle<STEP>(row0);
                at = row * (STEP / 2) + ((c >> 1 ^ swizzle<STEP / 2>(row)) << 4) + (c & 1) * 8;
            } else {  // rows of EXT elements: 8 chunks a piece of 64 bytes
                const int c = ((pos >> 2 ^ (row0 & 3)) << 2) | (pos & 3);
                at = row * (EXT * 2) + ((c >> 3 ^ (row & 3)) << 6) + (c & 7) * 8;
            }
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                uint32_t hi[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    hi[i] = w[i] & 0xFFFF0000u;
                    if (k < 2) w[i] = as_u(as_f(w[i]) - as_f(hi[i]));
                }
                *reinterpret_cast<u32x2*>(to + k * kPlane + at) =
                    (u32x2){__builtin_amdgcn_perm(hi[1], hi[0], 0x07060302u),
                            __builtin_amdgcn_perm(hi[3], hi[2], 0x07060302u)};
            }
        }
    }
    __device__ __forceinline__ void store_held(const Held& h, char* to) const {
        auto each = [&](auto any) {
#pragma unroll
            for (int q = 0; q < kLoads; ++q)
                *reinterpret_cast<u32x4*>(to + (q * THREADS + (int)threadIdx.x) * 16) =
                    decltype(any)::value ? shift_down(h.w[q], (LAYOUT == kAlong ? h.by : moved) * ES)
                                         : h.w[q];
        };
        if (__builtin_expect(LAYOUT == kAlong ? h.cut : edge, 0))
            each(std::true_type{});
        else
            each(std::false_type{});
    }
};

// A lane's fragment of rows [32 block, 32 block + 32) in the `sub`th 32 bytes of a step.
template <int DT, int LAYOUT, int EXT, int STEP>
__device__ __forceinline__ u32x4 fragment(const char* buf, int sub, int block) {
    constexpr int ES = Elem<DT>::kBytes, kRow = LAYOUT == kAlong ? STEP : EXT * ES;
    const int lane = (int)threadIdx.x & 63, hi = lane >> 5;
    if constexpr (LAYOUT == kAlong) {
        const int row = lane & 31;
        return *reinterpret_cast<const u32x4*>(buf + block * (32 * kRow) + row * kRow +
                                               ((2 * sub ^ (hi ^ swizzle<STEP>(row))) << 4));
    } else if constexpr (ES == 2) {
        // rows hi 8 + 0-3 and + 4-7 of 16; 64-byte piece c of row t is at c ^ (t & 3)
        const int t = (lane & 15) >> 2;
        const char* at = buf + (sub * 16 + hi * 8 + t) * kRow + ((block ^ t) << 6) +
                         (lane >> 4 & 1) * 32 + (lane & 3) * 8;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)at);
        const s16x4 up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(at + 4 * kRow));
        return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, up, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = *reinterpret_cast<const uint32_t*>(buf + (sub * 8 + hi * 4 + j) * kRow +
                                                      ((block * 2 + (lane >> 4 & 1) ^ j) << 6) +
                                                      (lane & 15) * 4);
        return v;
    }
}

// acc += a b^T over a quarter's k's.
template <int DT>
__device__ __forceinline__ f32x16 multiply(u32x4 a, u32x4 b, f32x16 acc) {
    if constexpr (DT == PTORED_BF16) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a),
                                                       __builtin_bit_cast(b8, b), acc, 0, 0, 0);
    } else if constexpr (DT == PTORED_F16) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a),
                                                      __builtin_bit_cast(h8, b), acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(as_f(a[j]), as_f(b[j]), acc, 0, 0, 0);
        return acc;
    }
}

// Waits until at most LEFT of this wave's loads are under way and its LDS
// accesses are done, then for the other waves.
// LEFT < 0: loads to registers, which the compiler waits for itself.
template <int LEFT>
__device__ __forceinline__ void landed() {
    if constexpr (LEFT >= 0)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LEFT) : "memory");
    else
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// C elements, 16 bytes of type DT, to or from a row of which `n` (at most C
// count) are left.
template <int DT, int C>
__device__ __forceinline__ void store_chunk(char* p, const float* v, int64_t n) {
    using E = Elem<DT>;
    static_assert(C == E::V, "a slot");
    if (__builtin_expect(n >= C, 1)) {
        *reinterpret_cast<u32x4_any*>(p) = E::narrow(v);
        return;
    }
#pragma unroll
    for (int i = 0; i < C - 1; ++i)
        if (i < n) E::store1(p + i * E::kBytes, v[i]);
}
template <int DT, int C>
__device__ __forceinline__ void add_chunk(const char* p, float* v, int64_t n) {
    using E = Elem<DT>;
    if (__builtin_expect(n >= C, 1)) {
        float w[C];
        E::widen(*reinterpret_cast<const u32x4_any*>(p), w);
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] += w[i];
        return;
    }
    float w[C];
#pragma unroll
    for (int i = 0; i < C - 1; ++i) w[i] = i < n ? E::load1(p + i * E::kBytes) : 0.0f;
#pragma unroll
    for (int i = 0; i < C - 1; ++i) v[i] += w[i];
}

// WM x WN waves of TM x TN blocks of 32 x 32; NS buffers of STEP bytes along k in
// the LDS.
// HOW: what comes to the LDS, and how.
enum : int {
    kDirect = 0,  // loaded straight into it
    kHeld = 1,    // through registers
    kSplit = 2,   // through registers, F32 as three bfloat16
    kShort = 3    // through registers, element by element
};
template <int WM, int WN, int TM, int TN, int STEP, int HOW>
constexpr int product_bytes() {  // a buffer in the LDS
    return (WM * TM + WN * TN) * 32 * STEP * (HOW == kSplit ? 3 : 2) / 2;
}
// Workgroup `id` of a product.  again(): the arguments where they are not kept in
// registers.
template <int DT, int KIND, int WM, int WN, int TM, int TN, int STEP, int NS, int HOW, typename F>
__device__ __forceinline__ void product_body(const ProductArgs& a, int id, char* lds, F again) {
    constexpr bool DIRECT = HOW == kDirect, SPLIT = HOW == kSplit;
    static_assert(!SPLIT || DT == PTORED_F32, "planes of F32");
    constexpr int kThreads = WM * WN * 64, BM = WM * TM * 32, BN = WN * TN * 32;
    constexpr bool kPair = KIND == kForward;  // a wave's lower blocks are the gate's, its upper ones the up's
    static_assert(!kPair || TN % 2 == 0, "as many gate's blocks as up's");
    static_assert(DIRECT || NS == 2, "registers hold the steps after the next");
    constexpr int LA = KIND == kWeight ? kAcross : kAlong, LB = KIND == kForward ? kAlong : kAcross;
    using A = Side<DT, LA, BM, STEP, kThreads, DIRECT, false>;
    using B = Side<DT, LB, BN, STEP, kThreads, DIRECT, kPair>;
    using E = Elem<DT>;
    // as multiplied: planes of bfloat16, each of half a step's bytes
    constexpr int FT = SPLIT ? (int)PTORED_BF16 : DT, P = SPLIT ? 3 : 1, kStep = SPLIT ? STEP / 2 : STEP;
    constexpr int kDepth = A::kDepth;
    constexpr int kPlaneA = SPLIT ? A::kPlane : A::kBytes, kPlaneB = SPLIT ? B::kPlane : B::kBytes;
    constexpr int kBytes = P * (kPlaneA + kPlaneB);
    constexpr int kLoads = DIRECT ? A::kLoads + B::kLoads : 0;  // of a step that barriers wait for
    static_assert((NS - 1) * kLoads <= 63, "as far as the hardware counts");
    constexpr int kCols = kPair ? BN / 2 : BN;  // of the output
    static_assert(kBytes == product_bytes<WM, WN, TM, TN, STEP, HOW>(), "the LDS");

    const int lane = (int)threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    // Workgroups go to the 8 dies in turn: each die gets consecutive tiles of
    // the order in which 4 rows of tiles advance together, so that its cache
    // serves most reads of both operands.
    const int tiles = a.tiles_m * a.tiles_n, total = tiles * a.outs * a.splits;
    {
        const int die = id % 8, each = total / 8, rest = total % 8;
        id = die * each + (die < rest ? die : rest) + id / 8;
    }
    const int split = id / (tiles * a.outs), in_split = id % (tiles * a.outs);
    const int which = in_split / tiles, tile = in_split % tiles;
    const int band = tile / (4 * a.tiles_n), band_rows = min(4, a.tiles_m - band * 4);
    const int in_band = tile - band * 4 * a.tiles_n;
    const int64_t m0 = (int64_t)(band * 4 + in_band % band_rows) * BM;
    const int64_t n0 = (int64_t)(in_band / band_rows) * kCols;

    // k's that a load looks at.
    auto remain = [&](int64_t left, bool any) { return any ? (int)min(left, (int64_t)1 << 20) : 0; };
    // Where the next load takes its step from.
    const int64_t per_pair = a.k > kDepth ? (a.k + kDepth - 1) / kDepth : 1;
    const int64_t all = KIND == kInput ? 2 * per_pair : per_pair;
    const int64_t first = split * a.steps_per_split;
    const int steps = (int)min(a.steps_per_split, all - first);
    // Tiles of few rows, whose time is that of the weights' way, begin at steps of
    // their own: rows are a pitch apart, and at one column all tiles would ask the
    // same memory channels.
    const int turn = KIND == kForward && BN == 64 ? (int)((uint32_t)id * 5 % (uint32_t)steps) : 0;
    int pair = 0, loaded = 0;  // the operands' pair; steps asked for
    int64_t left;
    const char *pa, *pb, *pb2;
    // (selected, not indexed: an array indexed by a register goes to scratch memory)
    int64_t a_ld = 0, b_ld = 0;
    auto begin = [&](int64_t step) {
        pair = KIND == kInput ? (int)(step / per_pair) : KIND == kWeight ? which : 0;
        const int64_t in = KIND == kInput ? step - pair * per_pair : step;
        const bool up = KIND != kForward && pair != 0, up_b = KIND == kInput && pair != 0;
        a_ld = up ? a.a_ld[1] : a.a_ld[0];
        b_ld = up_b ? a.b_ld[1] : a.b_ld[0];
        left = a.k - in * kDepth;
        pa = (up ? a.a[1] : a.a[0]) + (LA == kAlong ? m0 * a_ld + in * STEP
                                                    : in * kDepth * a_ld + m0 * E::kBytes);
        pb = (up_b ? a.b[1] : a.b[0]) + (LB == kAlong ? n0 * b_ld + in * STEP
                                                      : in * kDepth * b_ld + n0 * E::kBytes);
        pb2 = kPair ? a.b[1] + n0 * a.b_ld[1] + in * STEP : pb;
    };
    A sa;
    B sb;
    auto places = [&] {
        sa.init(m0, a.m, a_ld, a_ld);
        sb.init(n0, a.n, b_ld, kPair ? a.b_ld[1] : b_ld);
    };
    auto advance = [&] {
        ++loaded;
        left -= kDepth;
        if (KIND == kInput && left <= 0 && pair == 0) {
            begin(per_pair);
            places();
            return;
        }
        if (KIND == kForward && BN == 64 && loaded == steps - turn) {
            begin(first);
            return;
        }
        pa += LA == kAlong ? STEP : kDepth * a_ld;
        pb += LB == kAlong ? STEP : kDepth * b_ld;
        pb2 += STEP;
    };
    // extents of the rows that chunks lie in
    const int64_t ea = LA == kAlong ? a.k : a.m, eb = LB == kAlong ? a.k : a.n;
    // Registers: the steps after those in the LDS, two where they fit.
    constexpr int kSets = DIRECT || HOW == kShort ? 1 : TM * TN > 4 ? 1 : 2;
    typename A::Held ha[kSets];
    typename B::Held hb[kSets];
    auto hold = [&](auto which_set) {
        constexpr int set = decltype(which_set)::value;
        // past the last step the rows are over: zeros from nowhere
        const int n = remain(left, loaded < steps);
        sa.template load_held<HOW == kShort>(ha[set], pa, pa, n, ea);
        sb.template load_held<HOW == kShort>(hb[set], pb, pb2, n, eb);
        advance();
    };
    // The next step to a buffer, in two halves.  Past the last one zeros, from
    // nowhere, so that the loads under way stay countable.
    auto stage_a = [&](char* buf) {
        sa.load_direct(pa, pa, remain(left, loaded < steps), lds_address(buf));
    };
    auto stage_b = [&](char* buf) {
        sb.load_direct(pb, pb2, remain(left, loaded < steps), lds_address(buf) + A::kBytes);
        advance();
    };
    auto stage_held = [&](char* buf, auto which_set) {
        constexpr int set = decltype(which_set)::value;
        if constexpr (SPLIT) {
            sa.store_split(ha[set], buf);
            sb.store_split(hb[set], buf + P * kPlaneA);
        } else {
            sa.store_held(ha[set], buf);
            sb.store_held(hb[set], buf + A::kBytes);
        }
        hold(which_set);
    };
    using Set0 = std::integral_constant<int, 0>;
    using Set1 = std::integral_constant<int, kSets - 1>;

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = (f32x16)(0.0f);
    struct Fragments {
        u32x4 a[P][TM], b[P][TN];
    };
    auto read = [&](const char* buf, int sub, Fragments& f) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
                f.a[p][i] = fragment<FT, LA, BM, kStep>(buf + p * kPlaneA, sub, wm * TM + i);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                f.b[p][j] = fragment<FT, LB, BN, kStep>(
                    buf + P * kPlaneA + p * kPlaneB, sub,
                    kPair ? j / (TN / 2) * (WN * TN / 2) + wn * (TN / 2) + j % (TN / 2) : wn * TN + j);
        }
    };
    // Transposed: a lane's sums belong to one row of the output.  Of planes' products
    // those below 2^-22 of the largest are left out, the smallest taken first.
    auto products = [&](const Fragments& f) {
#pragma unroll
        for (int s = P - 1; s >= 0; --s)
#pragma unroll
            for (int p = 0; p <= s; ++p)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = multiply<FT>(f.b[p][j], f.a[s - p][i], acc[i][j]);
    };

    // The instructions of 32 bytes along k: the next fragments' reads between the first
    // products.  Left to itself the compiler puts each read right before its use.
    constexpr int kReadsA = LA == kAlong ? 1 : FT == PTORED_F32 ? 4 : 2;
    constexpr int kReadsB = LB == kAlong ? 1 : FT == PTORED_F32 ? 4 : 2;
    constexpr int kProducts = TM * TN * (FT == PTORED_F32 ? 4 : P * (P + 1) / 2);
    constexpr int kBetween = (P * (TM * kReadsA + TN * kReadsB) + kProducts - 1) / kProducts;
    auto order = [] {
#pragma unroll
        for (int i = 0; i < kProducts; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);         // matrix instruction
            __builtin_amdgcn_sched_group_barrier(0x100, kBetween, 0);  // LDS reads
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    begin(first + turn);
    places();
    if constexpr (DIRECT) {
#pragma unroll
        for (int b = 0; b < NS; ++b) {
            stage_a(lds + b * kBytes);
            stage_b(lds + b * kBytes);
        }
    } else {
        hold(Set0{});
        if constexpr (kSets == 2) hold(Set1{});
        stage_held(lds, Set0{});
        stage_held(lds + kBytes, Set1{});
    }
    landed<DIRECT ? (NS - 1) * kLoads : -1>();
    char *cur = lds, *last = lds;
    Fragments even, odd;
    read(cur, 0, even);
    auto step = [&](int s, auto set) {
        __builtin_amdgcn_sched_barrier(0);
        // b's half of what the last step began: with a's, the loads of all waves at
        // once keep the matrix cores waiting (3%)
        if (DIRECT && s > 0) stage_b(last);
        read(cur, 1, odd);
        products(even);
        order();
        if constexpr (kStep == 128) {
            read(cur, 2, even);
            products(odd);
            order();
            read(cur, 3, odd);
            products(even);
            order();
        }
        landed<DIRECT ? (NS - 2) * kLoads : -1>();
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (DIRECT)
            stage_a(cur);
        else
            stage_held(cur, set);
        last = cur;
        cur = cur == lds + (NS - 1) * kBytes ? lds : cur + kBytes;
        read(cur, 0, even);  // past the last step: zeros, never used
        products(odd);
        order();
    };
    if constexpr (kSets == 2) {
        for (int s = 0; s < steps; s += 2) {
            step(s, Set0{});
            if (s + 1 < steps) step(s + 1, Set1{});
        }
    } else {
        for (int s = 0; s < steps; ++s) step(s, Set0{});
    }
    landed<0>();  // the LDS may be another workgroup's after this

    // Register r of a block is column 8 (r / 4) + 4 (lane / 32) + r % 4 of row lane
    // % 32.  Each wave turns its blocks, 32 rows at a time, in LDS of its own, so
    // that its lanes store whole pieces of rows: from the registers a store reaches
    // 32 rows, 32 bytes of each.  A row's pieces of 16 bytes change places with
    // the row, so that a piece's rows lie in different banks.
    constexpr int kBlocks = kPair ? TN / 2 : TN, kPitch = kBlocks * 32;
    auto placed = [](int row, int col) {
        return row * kPitch + ((col >> 2 ^ (kBlocks == 1 ? row >> 1 & 7 : row & 15)) << 2);
    };
    constexpr int kArea = 32 * kPitch;
    static_assert(WM * WN * (kPair ? 2 : 1) * kArea * 4 <= NS * kBytes, "room for it");
    float* const area = reinterpret_cast<float*>(lds) + wave * ((kPair ? 2 : 1) * kArea);
    // the arguments read again: nothing that only this end needs stays in registers
    // over the steps
    const ProductArgs& z = again();
    const int64_t tile_col = n0 + wn * (kBlocks * 32);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t tile_row = m0 + (wm * TM + i) * 32;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4*>(area + j / kBlocks * kArea +
                                          placed(lane & 31, j % kBlocks * 32 + q * 8 + (lane >> 5) * 4)) =
                    (f32x4){acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                            acc[i][j][4 * q + 3]};
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        // f(row, column, columns left, sums of C columns in each area) of what is inside
        auto pieces = [&](auto chunk, auto f) {
            constexpr int C = decltype(chunk)::value, kPerRow = kBlocks * 32 / C, kAtOnce = 64 / kPerRow;
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += kAtOnce) {
                const int r = r0 + lane / kPerRow, c = lane % kPerRow * C;
                const int64_t row = tile_row + r, col = tile_col + c;
                if (row >= z.m || col >= z.n) continue;
                float v[C], w[C];
#pragma unroll
                for (int k = 0; k < C; k += 4) {
                    const f32x4 x = *reinterpret_cast<const f32x4*>(area + placed(r, c + k));
                    const f32x4 y = kPair ? *reinterpret_cast<const f32x4*>(area + kArea + placed(r, c + k)) : x;
#pragma unroll
                    for (int l = 0; l < 4; ++l) {
                        v[k + l] = x[l];
                        w[k + l] = y[l];
                    }
                }
                f(row, col, z.n - col, v, w);
            }
        };
        using Narrow = std::integral_constant<int, E::V>;
        using Wide = std::integral_constant<int, 4>;
        if (z.splits > 1) {
            // ws_ld holds whole vectors of 4, which the join reads
            pieces(Wide{}, [&](int64_t row, int64_t col, int64_t, float* v, float* w) {
                const int64_t outs = kPair ? 2 : z.outs;
                float* p = z.ws + (((int64_t)split * outs + which) * z.m + row) * z.ws_ld + col;
                *reinterpret_cast<f32x4*>(p) = (f32x4){v[0], v[1], v[2], v[3]};
                if (kPair) *reinterpret_cast<f32x4*>(p + z.m * z.ws_ld) = (f32x4){w[0], w[1], w[2], w[3]};
            });
        } else if constexpr (kPair) {
            pieces(Narrow{}, [&](int64_t row, int64_t col, int64_t n, float* g, float* u) {
                constexpr int C = E::V;
                float y[C];
#pragma unroll
                for (int e = 0; e < C; ++e) y[e] = activation<DT>(z.activation, g[e]) * u[e];
                store_chunk<DT, C>(z.out[0].p + row * z.out[0].ld + col * E::kBytes, y, n);
                if (z.gate.p) store_chunk<DT, C>(z.gate.p + row * z.gate.ld + col * E::kBytes, g, n);
                if (z.up.p) store_chunk<DT, C>(z.up.p + row * z.up.ld + col * E::kBytes, u, n);
            });
        } else {
            const Mat out = which ? z.out[1] : z.out[0];
            if (z.out_f32) {
                pieces(Wide{}, [&](int64_t row, int64_t col, int64_t n, float* v, float*) {
                    char* p = out.p + row * out.ld + col * 4;
                    if (z.accumulate) add_chunk<PTORED_F32, 4>(p, v, n);
                    store_chunk<PTORED_F32, 4>(p, v, n);
                });
            } else {
                pieces(Narrow{}, [&](int64_t row, int64_t col, int64_t n, float* v, float*) {
                    char* p = out.p + row * out.ld + col * E::kBytes;
                    if (z.accumulate) add_chunk<DT, E::V>(p, v, n);
                    store_chunk<DT, E::V>(p, v, n);
                });
            }
        }
    }
}

template <int DT, int KIND, int WM, int WN, int TM, int TN, int STEP, int NS, int HOW>
__global__ __launch_bounds__(WM* WN * 64) void product_kernel(const ProductArgs a) {
    __shared__ __attribute__((aligned(1024))) char lds[NS * product_bytes<WM, WN, TM, TN, STEP, HOW>()];
    product_body<DT, KIND, WM, WN, TM, TN, STEP, NS, HOW>(
        a, (int)blockIdx.x, lds, []() -> const ProductArgs& { return args_again<ProductArgs>(); });
}

// The input's gradient and the weights' in one launch, in tiles of 128: either
// alone leaves compute units idle where the matrices are small (5467 tokens, 655
// columns, 324 features, bf16: 23 and 22 us one after the other).  8 waves, two
// workgroups a compute unit (2048 x 1001 x 1003 54 us in 4 waves, 47).
template <int DT, int HOW>
__global__ __launch_bounds__(512) void product_both_kernel(const ProductPair p) {
    __shared__ __attribute__((aligned(1024))) char lds[2 * product_bytes<2, 2, 2, 2, 128, HOW>()];
    const int id = (int)blockIdx.x;
    if (id < p.first)
        product_body<DT, kWeight, 4, 2, 1, 2, 128, 2, HOW>(
            p.weight, id, lds, []() -> const ProductArgs& { return args_again<ProductPair>().weight; });
    else
        product_body<DT, kInput, 4, 2, 1, 2, 128, 2, HOW>(
            p.input, id - p.first, lds, []() -> const ProductArgs& { return args_again<ProductPair>().input; });
}

// out (+)= the splits' sums, or the forward pass's outputs from them.  A workgroup
// takes 64 times 4 columns of a row, 4 threads each for every fourth split,
// joined in the LDS in a fixed order.
constexpr int kJoinLanes = 64, kJoinGroups = 4;
template <int DT, int KIND>
__device__ __forceinline__ void product_join(const ProductArgs& a) {
    using E = Elem<DT>;
    constexpr int kSums = KIND == kForward ? 2 : 1;  // g and u
    __shared__ f32x4 part[kSums][kJoinGroups][kJoinLanes];
    const int lane = (int)threadIdx.x % kJoinLanes, group = (int)threadIdx.x / kJoinLanes;
    const int64_t col = ((int64_t)blockIdx.x * kJoinLanes + lane) * 4;
    const int64_t rows = a.m * (KIND == kForward ? 1 : a.outs), step = rows * kSums * a.ws_ld;
    for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
        f32x4 sum[kSums] = {};
        if (col < a.n) {
            const float* ws = a.ws + row * a.ws_ld + col;
#pragma unroll 4
            for (int s = group; s < a.splits; s += kJoinGroups)
#pragma unroll
                for (int k = 0; k < kSums; ++k)
                    sum[k] += *reinterpret_cast<const f32x4*>(ws + s * step + k * rows * a.ws_ld);
        }
#pragma unroll
        for (int k = 0; k < kSums; ++k) part[k][group][lane] = sum[k];
        __syncthreads();
        if (group == 0 && col < a.n) {
            const bool second = KIND != kForward && row >= a.m;
            const int64_t r = second ? row - a.m : row;
            const Mat out = second ? a.out[1] : a.out[0];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (col + i >= a.n) continue;
                float v[kSums];
#pragma unroll
                for (int k = 0; k < kSums; ++k)
                    v[k] = (part[k][0][lane][i] + part[k][1][lane][i]) +
                           (part[k][2][lane][i] + part[k][3][lane][i]);
                if constexpr (KIND == kForward) {
                    const int64_t at = (col + i) * E::kBytes;
                    E::store1(out.p + r * out.ld + at, activation<DT>(a.activation, v[0]) * v[1]);
                    if (a.gate.p) E::store1(a.gate.p + r * a.gate.ld + at, v[0]);
                    if (a.up.p) E::store1(a.up.p + r * a.up.ld + at, v[1]);
                } else if (a.out_f32) {
                    float* p = reinterpret_cast<float*>(out.p + r * out.ld) + col + i;
                    *p = a.accumulate ? *p + v[0] : v[0];
                } else {
                    char* p = out.p + r * out.ld + (col + i) * E::kBytes;
                    if (a.accumulate) v[0] += E::load1(p);
                    E::store1(p, v[0]);
                }
            }
        }
        __syncthreads();
    }
}

template <int DT, int KIND>
__global__ __launch_bounds__(kJoinLanes* kJoinGroups) void product_join_kernel(const ProductArgs a) {
    product_join<DT, KIND>(a);
}
// Those of either product that has splits.
template <int DT>
__global__ __launch_bounds__(kJoinLanes* kJoinGroups) void product_both_join_kernel(const ProductPair p) {
    if (blockIdx.z == 0)
        product_join<DT, kWeight>(p.weight);
    else
        product_join<DT, kInput>(p.input);
}

// The joining kernel's workgroups.
inline dim3 product_joins(const ProductArgs& a, int kind) {
    const int64_t rows = a.m * (kind == kForward ? 1 : a.outs);
    return dim3((uint32_t)((a.n + 4 * kJoinLanes - 1) / (4 * kJoinLanes)),
                (uint32_t)(rows < 32768 ? rows : 32768));
}

template <int DT>
int product_both_launch(const ProductPair& p, hipStream_t stream) {
    void* args[] = {const_cast<ProductPair*>(&p)};
    const ProductArgs &w = p.weight, &x = p.input;
    const void* k = w.direct && x.direct ? reinterpret_cast<const void*>(product_both_kernel<DT, kDirect>)
                                         : reinterpret_cast<const void*>(product_both_kernel<DT, kHeld>);
    const uint32_t grid = (uint32_t)p.first + (uint32_t)x.tiles_m * (uint32_t)x.tiles_n * (uint32_t)x.splits;
    if (hipLaunchKernel(k, dim3(grid), dim3(512), args, 0, stream) != hipSuccess) return kFailed;
    if (w.splits > 1 && x.splits > 1) {
        const dim3 a = product_joins(w, kWeight), b = product_joins(x, kInput);
        const dim3 both(a.x > b.x ? a.x : b.x, a.y > b.y ? a.y : b.y, 2);
        return hipLaunchKernel(reinterpret_cast<const void*>(product_both_join_kernel<DT>), both,
                               dim3(kJoinLanes * kJoinGroups), args, 0, stream) == hipSuccess
                   ? kOk
                   : kFailed;
    }
    const bool input = x.splits > 1;
    if (!input && w.splits == 1) return kOk;
    void* one[] = {const_cast<ProductArgs*>(input ? &x : &w)};
    k = input ? reinterpret_cast<const void*>(product_join_kernel<DT, kInput>)
              : reinterpret_cast<const void*>(product_join_kernel<DT, kWeight>);
    return hipLaunchKernel(k, input ? product_joins(x, kInput) : product_joins(w, kWeight),
                           dim3(kJoinLanes * kJoinGroups), one, 0, stream) == hipSuccess
               ? kOk
               : kFailed;
}

template <int DT, int KIND>
int product_launch(const ProductArgs& a, hipStream_t stream) {
    void* args[] = {const_cast<ProductArgs*>(&a)};
    const void* k = nullptr;
    int threads = 256;
    if (a.shape >= kFew16) {
        if constexpr (KIND != kForward) return kFailed;
        const int rc = few_launch<DT>(a, stream);
        if (rc != kOk) return rc;
    } else {
        if (a.shape == kTile32x128) {
            if constexpr (KIND == kInput) {
                k = reinterpret_cast<const void*>(product_kernel<DT, KIND, 1, 4, 1, 1, 128, 2, kHeld>);
                if (a.direct) {
                    if constexpr (DT != PTORED_F32) return kFailed;
                    else k = reinterpret_cast<const void*>(product_kernel<DT, KIND, 1, 4, 1, 1, 128, 4, kDirect>);
                }
            } else {
                return kFailed;
            }
        } else if (a.shape == kTile64x128) {
            if constexpr (KIND == kWeight) return kFailed;
            else k = a.direct ? reinterpret_cast<const void*>(product_kernel<DT, KIND, 2, 2, 1, 2, 128, 3, kDirect>)
                              : reinterpret_cast<const void*>(product_kernel<DT, KIND, 2, 2, 1, 2, 128, 2, kHeld>);
        } else if (a.shape == kTileSplit) {
            threads = 512;
            if constexpr (DT != PTORED_F32) return kFailed;
            else k = reinterpret_cast<const void*>(product_kernel<DT, KIND, 4, 2, 2, 2, 128, 2, kSplit>);
        } else if (a.shape == kTileShort) {
            k = reinterpret_cast<const void*>(product_kernel<DT, KIND, 2, 2, 2, 2, 128, 2, kShort>);
        } else if (!a.direct) {
            // 8 waves hide more of the way through registers; the weights' reads across
            // rows, of both operands, then cost more (501 x 1003 x 2501 f16 24.0, 20.1 us;
            // 512 x 4095 x 8193 input's gradient 132, 125, the weights' 129, 133)
            constexpr bool kMany = KIND != kWeight;
            threads = kMany ? 512 : 256;
            k = reinterpret_cast<const void*>(product_kernel<DT, KIND, kMany ? 4 : 2, 2, kMany ? 1 : 2, 2, 128, 2, kHeld>);
            if constexpr (DT != PTORED_F32) {
                if (a.shape == kTile256) {
                    threads = 512;
                    k = reinterpret_cast<const void*>(product_kernel<DT, KIND, 2, 4, 4, 2, 128, 2, kHeld>);
                }
            }
        } else if (a.shape == kTile128) {
            k = reinterpret_cast<const void*>(product_kernel<DT, KIND, 2, 2, 2, 2, 128, 2, kDirect>);
        } else if (a.shape == kTile128Deep) {
            // one workgroup a compute unit: two waves for each of its matrix cores (512
            // x 1536 x 4096 bf16 21.8, 20.0 us)
            threads = 512;
            k = reinterpret_cast<const void*>(product_kernel<DT, KIND, 4, 2, 1, 2, 128, 4, kDirect>);
        } else if (a.shape == kTile256) {
            threads = 512;
            if constexpr (DT == PTORED_F32) return kFailed;
            else k = reinterpret_cast<const void*>(product_kernel<DT, KIND, 2, 4, 4, 2, 128, 2, kDirect>);
        } else if (a.shape == kTile64) {
            threads = 128;
            if constexpr (KIND != kForward || DT == PTORED_F32) return kFailed;
            else k = reinterpret_cast<const void*>(product_kernel<DT, KIND, 2, 1, 1, 2, 128, 8, kDirect>);
        } else {
            if constexpr (KIND != kForward) return kFailed;
            else k = reinterpret_cast<const void*>(product_kernel<DT, KIND, 4, 1, 1, 2, 128, 6, kDirect>);
        }
        const uint32_t grid = (uint32_t)a.tiles_m * (uint32_t)a.tiles_n * (uint32_t)(a.outs * a.splits);
        if (hipLaunchKernel(k, dim3(grid), dim3((uint32_t)threads), args, 0, stream) != hipSuccess)
            return kFailed;
    }
    if (a.splits == 1) return kOk;
    return hipLaunchKernel(reinterpret_cast<const void*>(product_join_kernel<DT, KIND>), product_joins(a, KIND),
                           dim3(kJoinLanes * kJoinGroups), args, 0, stream) == hipSuccess
               ? kOk
               : kFailed;
}

}  // namespace step
}  // namespace ptored
