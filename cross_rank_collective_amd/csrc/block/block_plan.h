// block_plan.h -- what the host code hands to the kernels of the
// block-boundary operators, and the launch functions (one per element type,
// each in a unit of its own, block_ops.hip).
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "ptored_block.h"

namespace ptored {
namespace block {

// A matrix as the kernels address it: a null base means "not there".
struct Mat {
    char* p;
    int64_t ld;  // bytes from one row to the next
};

// A packed matrix; q null means "not there".
struct Kept {
    int8_t* q;
    int64_t q_ld;
    uint8_t* s;
    int64_t s_ld;
};

struct NormArgs {
    const char* part[PTORED_MAX_RANKS];
    int64_t part_ld;  // bytes
    int64_t rows;
    Mat x, x_out, z, h, gate;
    Kept kh, kx, kz;
    const char *w1, *w2;
    float *r1, *r2;
    int64_t rows_per_gate;
    int32_t nranks, cols, w_f32;
    float offset, alpha, beta, eps, inv_cols;
};

// Gate rows within a chunk of the backward pass.
enum : int {
    kOneGate = 0,   // one, or there is no gate
    kEachGate = 1,  // every row has its own
    kSomeGates = 2  // several, of any length
};

struct GradArgs {
    int64_t rows;
    Mat dz, dxo, x, h, dx, dh, gate, dgate;
    Kept kx, kh;
    const char *w1, *w2;
    const float *r1, *r2;
    float* ws;              // partial sums: [chunk][which][ws_pitch]
    char *dw1, *dw2;
    // rows are cut into units of unit_rows, each unit into chunks_per_unit
    // chunks of at most chunk_rows rows: chunk j of a unit begins with its row
    // j chunk_first and takes every row_step-th
    int64_t unit_rows, chunks_per_unit, chunk_rows, chunk_first, row_step;
    int64_t chunks;
    int64_t gate_rows;
    int64_t rows_per_gate;
    int64_t ws_pitch;     // the columns, rounded up to whole vectors of 4
    int32_t chunk_gates;  // kOneGate, kEachGate or kSomeGates
    int32_t gate_direct;  // 1: chunks hold whole gate rows and write their gradients
    int32_t gate_joined;  // 1: the gate's gradients come from the chunks' A
    int32_t gate_units;   // gate rows from one unit to the next: 1, or 0 with one in all
    int32_t ws_slots;     // partial rows per chunk: A or dw1, and dw2
    int32_t slot_w1, slot_w2;  // which of them; -1: none
    int32_t cols, w_f32;
    float offset, alpha, beta, inv_cols;
};

// How the backward pass cuts its rows: a chunk is what one workgroup walks,
// keeping the column sums in registers.  With a gate the chunks never
// straddle two gate rows unless they hold whole ones.
struct GradSplit {
    int64_t unit_rows, chunks_per_unit, chunk_rows, chunk_first, row_step, chunks;
    int32_t gate_direct;
};

struct PackArgs {
    Mat x;
    Kept k;
    int64_t rows;
    int32_t cols;
};

// The weight gradient's workgroups.
enum : int {
    kWgradTile = 0,  // tiles of 128 x 128 (f32: 128 x 256), 64 tokens a step (f32: 32)
    kWgradWide = 1,  // 256 x 256, 32 tokens a step; not f32
    kWgradFew = 2    // 128 x 128 of a matrix with rows shorter than a chunk
};

struct WgradArgs {
    const char* dy;
    int64_t dy_ld;  // bytes
    Kept x;
    char* dw;
    int64_t dw_ld;  // bytes
    float* ws;      // [split][outs][ws_ld] partial sums when splits > 1
    int64_t ws_ld;  // the columns, rounded up to whole vectors of 4
    int64_t rows;
    int64_t rows_per_split;  // a multiple of the kernel's step
    int32_t outs, cols;
    int32_t splits;
    int32_t dw_f32, accumulate;
    int32_t tiles_m, tiles_n;
    int32_t shape;  // kWgradTile, kWgradWide or kWgradFew
};

enum : int { kOk = 0, kFailed = 1 };

// T = f32, bf16, f16
#define PTORED_BLOCK_LAUNCHES(T)                            \
    int norm_##T(const NormArgs&, hipStream_t);             \
    int grad_##T(const GradArgs&, hipStream_t);             \
    int pack_##T(const PackArgs&, hipStream_t);             \
    int unpack_##T(const PackArgs&, hipStream_t);           \
    int wgrad_##T(const WgradArgs&, hipStream_t);
PTORED_BLOCK_LAUNCHES(f32)
PTORED_BLOCK_LAUNCHES(bf16)
PTORED_BLOCK_LAUNCHES(f16)
#undef PTORED_BLOCK_LAUNCHES

}  // namespace block
}  // namespace ptored
