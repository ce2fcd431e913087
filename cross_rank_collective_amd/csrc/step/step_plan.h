// step_plan.h -- what the host code hands to the kernels of the step's
// operators, and the launch functions (one per element type where they depend
// on one, each in a unit of its own, step_ops.hip).
#pragma once

#include "block/block_plan.h"
#include "ptored_step.h"

namespace ptored {
namespace step {

using block::kFailed;
using block::kOk;
using block::Mat;

struct LayerNormArgs {
    const char* part[PTORED_MAX_RANKS];
    int64_t part_ld;  // bytes
    int64_t rows;
    Mat x, x_out, z;
    const char *w, *b;
    float *mean, *rstd;
    int32_t nranks, cols, w_f32;
    float eps, inv_cols;
};

struct LayerGradArgs {
    int64_t rows;
    Mat dz, dxo, x, dx;
    const char* w;
    const float *mean, *rstd;
    float* ws;         // partial sums: [chunk][dw, db][ws_pitch]
    char *dw, *db;
    int64_t chunks;    // workgroups; chunk c takes rows c, c + chunks, ...
    int64_t ws_pitch;  // the columns, rounded up to whole vectors of 4
    int32_t cols, w_f32;
    float inv_cols;
};

// Layouts of a product's operands: the sum's index along rows (k consecutive)
// or across them (k is the row).
enum : int { kAlong = 0, kAcross = 1 };

// The products of the feed-forward block.
enum : int {
    kForward = 0,  // f(x Wg^T) (x Wu^T): both operands along
    kInput = 1,    // dg Wg + du Wu: dg along, weights across
    kWeight = 2    // dg^T x and du^T x: both across
};

struct ProductArgs {
    // kForward: x; Wg, Wu.  kInput: dg, du; Wg, Wu.  kWeight: dg, du; x.
    const char *a[2], *b[2];
    int64_t a_ld[2], b_ld[2];  // bytes
    int64_t m, n, k;           // kForward: n features of each weight; kInput: k of each pair
    Mat out[2];                // kForward: y; kInput: dx; kWeight: dWg, dWu
    Mat gate, up;              // kForward: what is kept
    float* ws;                 // [split][out][m][ws_ld] partial sums when splits > 1
                               // (kForward: g and u as two outs)
    int64_t ws_ld;             // n, rounded up to whole vectors of 4
    int64_t steps_per_split;
    int32_t tiles_m, tiles_n, splits;
    int32_t outs;        // kWeight: products, 1 or 2
    int32_t waves;       // kFew16 to kFew64: of a workgroup
    int32_t out_f32, accumulate, activation;
    int32_t shape;       // a tile of kShapes
    int32_t direct;      // every row and column range is whole aligned chunks
};

// Both gradients of a call in one launch, in tiles kTile128: the weights'
// workgroups first.  A split product's partial sums are behind the other's.
struct ProductPair {
    ProductArgs weight, input;
    int32_t first;  // workgroups of the weights'
};

// Tiles of the products.
enum : int {
    kTile128 = 0,      // 128 x 128, 4 waves, two workgroups a compute unit (8 waves where not
                       // aligned, but for kWeight alone, and in launches of both gradients)
    kTile128Deep = 1,  // 8 waves, loads three steps ahead, one a compute unit; aligned
    kTile256 = 2,      // 256 x 256, 8 waves; 16-bit types
    kTile64 = 3,       // kForward: 64 tokens x 32 features, 2 waves; 16-bit types, aligned
    kTile128x32 = 4,   // kForward: 128 tokens x 32 features, 4 waves; aligned
    kTile32x128 = 5,   // kInput: 32 tokens x 128 columns, 4 waves; F32, and 16-bit types where not aligned
    kTile64x128 = 6,   // 64 x 128, 4 waves, two or (not aligned) three workgroups a compute unit
    kTileSplit = 7,    // 256 x 128, 8 waves, F32 as three bfloat16
    kTileShort = 8,    // 128 x 128, 4 waves, rows that do not hold 16 bytes
    kFew16 = 9,        // kForward of up to 16 tokens
    kFew32 = 10,       // 32 tokens; F32
    kFew64 = 11        // 64 tokens; F32
};
constexpr int kStepBytes = 128;  // of each row along k that a step takes

struct SlopeArgs {  // dg and du
    Mat dy, gate, up, dgate, dup;
    int64_t rows, cols;
    int32_t activation;
};

// Gradients of a call.  An entry is rows x cols elements, cut into chunks of
// kGradChunk elements, or of as many slots of 16 bytes where there are several
// rows (each with its last slot perhaps partly filled).
constexpr int kGradChunk = 2048;
constexpr int kGradPerUnit = 8;                   // workgroups at once on a compute unit
constexpr int kGradGroups = 256 * kGradPerUnit;   // and on the chip
constexpr int kGradEntries = 72;                  // that a launch's arguments hold
constexpr int64_t kGradMost = int64_t(1) << 40;   // elements of a gradient of one row
constexpr int64_t kGradPitch = int64_t(1) << 27;  // and from one row to the next of several
inline __host__ __device__ int64_t grad_chunks(int64_t rows, int64_t cols, int dtype) {
    if (rows == 1) return (cols + kGradChunk - 1) / kGradChunk;
    const int64_t slot = dtype == PTORED_F32 ? 4 : 8, chunk = kGradChunk / slot;
    return (rows * ((cols + slot - 1) / slot) + chunk - 1) / chunk;
}
struct GradEntry {
    const char* data;
    char* out;
    int64_t cols;
    int32_t rows;
    int32_t ld, out_ld;  // elements
    int32_t first;       // the entry's first chunk
    int32_t type;        // dtype | out_dtype << 8
    int32_t unused;
};
struct GradList {
    GradEntry e[kGradEntries];
    const GradEntry* table;  // all entries in the workspace where they are more, or null
    int32_t count, chunks;   // entries and chunks of all
    int32_t groups;          // workgroups
    double* sums;            // partial sums, one for each workgroup
    const double* all;       // those to be joined, or null: `norm` is given
    int32_t all_count;
    float* norm;
    float max_norm;
};

// More entries than that on their way to a table in the workspace, packed: one
// slot of a single run, two of rows with gaps.
constexpr int kGradSlots = 192;
struct GradPack {
    GradEntry* table;               // where this launch's entries go
    int32_t first;                  // their first chunk
    int32_t slots;
    uint32_t heads[kGradSlots / 32];  // slots that begin an entry
    // an entry's first slot: address | elements of a row >> 32 << 48 | type << 56
    // (3 bits, type = dtype + 3 where the output is wider) | 1 << 59 with a
    // second slot; the second: rows | pitch << 32
    uint64_t data[kGradSlots];
    uint64_t out[kGradSlots];   // address; the output's pitch
    uint32_t cols[kGradSlots];  // elements of a row, low half
};

int grad_table(const GradPack&, hipStream_t);
int grad_sums(const GradList&, hipStream_t);
int grad_join(const GradList&, hipStream_t);
int grad_scale(const GradList&, hipStream_t);

// T = f32, bf16, f16
#define PTORED_STEP_LAUNCHES(T)                              \
    int layer_norm_##T(const LayerNormArgs&, hipStream_t);   \
    int layer_grad_##T(const LayerGradArgs&, hipStream_t);   \
    int product_forward_##T(const ProductArgs&, hipStream_t);\
    int product_input_##T(const ProductArgs&, hipStream_t);  \
    int product_weight_##T(const ProductArgs&, hipStream_t); \
    int product_both_##T(const ProductPair&, hipStream_t);   \
    int product_slope_##T(const SlopeArgs&, hipStream_t);
PTORED_STEP_LAUNCHES(f32)
PTORED_STEP_LAUNCHES(bf16)
PTORED_STEP_LAUNCHES(f16)
#undef PTORED_STEP_LAUNCHES

}  // namespace step
}  // namespace ptored
