// step_host.cpp -- C ABI of the step's operators: argument checks, work
// splits, launches.
//
// Every argument check runs before the first HIP call, so every error status
// is reachable without a GPU.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <memory>
#include <new>

#include "block/block_checks.hpp"
#include "step_plan.h"

namespace ptored {
namespace step {
namespace {

using namespace block;

// ---------------------------------------------------------------- layer norm

bool layer_valid(const ptored_layer_norm_params* p) {
    return p != nullptr && shape_ok(p->rows, p->cols);
}
bool layer_supported(const ptored_layer_norm_params& p) {
    return float_type(p.dtype) && (p.weight_dtype == PTORED_F32 || p.weight_dtype == p.dtype) &&
           p.cols <= PTORED_BLOCK_MAX_COLS;
}

// Workgroups of the backward pass: as many as the chip holds at once, but with
// work for all compute units none takes fewer than 5 rows, whose partial rows
// (8 bytes a column) would weigh as much as the rows' own data.
int64_t layer_chunks(int64_t rows, int64_t cols, int dtype) {
    if (rows == 0 || cols == 0) return 0;
    const int64_t slot = dtype == PTORED_F32 ? 4 : 8, room = dtype == PTORED_F32 ? 20 : 16;
    const int64_t waves = std::min<int64_t>(16, (cols + 64 * slot - 1) / (64 * slot));
    const int64_t target = 256 * (room / waves);
    const int64_t per = std::max((rows + target - 1) / target,
                                 std::min<int64_t>(5, (rows + 255) / 256));
    return (rows + per - 1) / per;
}
// Columns of a partial row: whole vectors of 4.
int64_t pitch_of(int64_t cols) { return (cols + 3) / 4 * 4; }
int64_t layer_workspace(int64_t chunks, int64_t cols) { return chunks * 2 * pitch_of(cols) * 4; }

// ---------------------------------------------------------------- feed-forward

bool ffn_valid(const ptored_ffn_params* p) {
    return p != nullptr && shape_ok(p->rows, p->cols) && shape_ok(p->rows, p->wide) &&
           shape_ok(p->wide, p->cols);
}
bool ffn_supported(const ptored_ffn_params& p) {
    return float_type(p.dtype) && p.activation >= PTORED_SILU && p.activation <= PTORED_GELU_TANH;
}
// A matrix whose tiles' offsets fit 32 bits.
bool pitch_supported(const ptored_rows& r, int64_t rows, int es) {
    return r.data == nullptr || rows <= 1 || r.ld <= PTORED_FFN_MAX_PITCH / es;
}
bool widths_supported(const ptored_ffn_params& p, int es) {
    return p.cols <= PTORED_FFN_MAX_PITCH / es && p.wide <= PTORED_FFN_MAX_PITCH / es;
}
// An operand as the kernels address it: a single row has no pitch of its own.
ptored_rows operand(const ptored_rows& r, int64_t rows, int64_t cols) {
    return {r.data, rows > 1 ? r.ld : cols};
}
// Rows that start at multiples of 16 bytes and hold whole chunks of 16.
bool direct_of(const ptored_rows& r, int64_t rows, int64_t cols, int es) {
    return reinterpret_cast<uintptr_t>(r.data) % 16 == 0 && cols * es % 16 == 0 &&
           (rows <= 1 || r.ld * es % 16 == 0);
}

struct ProductShape {
    int64_t tiles_m, tiles_n, splits, steps_per_split;
    int shape, waves;
    double us;  // estimated
};

constexpr int64_t kMaxTiles = int64_t(1) << 22;

// Whether an operand's rows are shorter than 16 bytes.
bool short_rows(int kind, int64_t m, int64_t n, int64_t k, int es) {
    return (kind == kForward ? k : std::min(n, kind == kInput ? k : m)) * es < 16;
}

// A tile's rows and columns of the output, and its time: base + step us for each
// of its steps, `slots` tiles at once, or base + alone where no compute unit has
// two (fits to 16 to 8192 tokens, 512 to 4096 columns and 640 to 16384 features).
struct TileCost {
    int shape;
    int64_t rows, cols, slots;
    double base, alone, step;
};

// many: 8 waves.
TileCost tile128(int64_t half, bool f32, bool direct, bool many) {
    if (direct) return {kTile128, 128, 128 / half, 512, 5, f32 ? 2.0 : 1.0, f32 ? 3.9 : 1.1};
    return {kTile128, 128, 128 / half, 512, 5, f32 ? 2.0 : many ? 1.0 : 1.15, f32 ? 3.9 : 1.35};
}

// Tiles and splits of a product, by estimated time; for kInput k is that of each
// of the two pairs.  Splits share a tile's steps among several workgroups, each
// of which writes its sums in 32 bits, which a second kernel reads again: 4 us
// and the bytes at 4 TB/s.
//
// Measured (forward, bf16, D = 4096, F = 8192, us): 1 token 25 with kFew16, 60 in
// tiles of 128; 32 tokens 32 with kTile64, 37 as kFew32 in that type; 64: 34, 41;
// 128: 37 with kTile128x32, 68 in tiles of 128; in tiles of 128, the same with loads
// further ahead, and 256: 192 tokens 70, 45, 103; 512: 85, 101, 107; 1024: 159,
// 178, 122.  Rows that do not start at multiples of 16 bytes (D = 4095, F = 8193):
// 64 tokens 80 in tiles of 128, 157 as kFew64; 2048 tokens 460, in tiles of 256
// 400.  In 32 bits kTile64's two waves are not enough for its products (64 tokens
// 149, kFew64 80).
ProductShape product_shape(int kind, int64_t m, int64_t n, int64_t k, int outs, int dtype,
                           bool direct) {
    const bool f32 = dtype == PTORED_F32;
    const int es = esize_of(dtype);
    const int64_t depth = kStepBytes / es;
    const int64_t steps = std::max<int64_t>(1, (k + depth - 1) / depth) * (kind == kInput ? 2 : 1);
    ProductShape s{};
    s.splits = 1;
    s.steps_per_split = steps;
    if (m == 0 || n == 0) return s;
    // what a split writes and the join reads
    const double join = (double)(kind == kForward ? 2 : outs) * (double)m * (double)n * 8 / 4e6;
    double best = -1;
    if (kind == kForward && (m <= 16 || (f32 && m <= 64)) && k * es >= 16) {
        s.shape = m <= 16 ? kFew16 : m <= 32 ? kFew32 : kFew64;
        s.tiles_m = 1;
        const int64_t features = s.shape == kFew64 ? 32 : 16;
        s.tiles_n = (n + features - 1) / features;
        // A compute unit takes 37 bytes of the weights a ns, the memory 5500 for all,
        // the same for each unit that still has a workgroup: those that have one more
        // than the others go on alone.  (1 token, f32, 5440 columns: 4096 features
        // 35 us, 5056 56 in 316 workgroups, 6144 57, 8192 63; 8192 columns x 2048
        // features, 128 workgroups: 19.)  More than 16 tokens in F32 are bound by the
        // products, 20 and 15.5 bytes a ns, and few features by tiles with splits
        // (47 tokens, us, kFew64 and tiles: 1792 columns x 256 26, 13; 1024 x 2048 24,
        // 16; 4096 x 8192 76, 86; 32 tokens, kFew32: 1792 x 256 18, 13; 1536 x 4096
        // 17, 23).
        const double rate = s.shape == kFew16 ? 37e3 : s.shape == kFew32 ? 20e3 : 15.5e3;
        const double base = s.shape == kFew16 ? 0.0 : 6.0;
        const int64_t units = k * es / 256;  // that waves share
        for (int64_t splits = 1; splits <= 16 && (splits == 1 || units >= 8 * splits); splits *= 2) {
            const double bytes = 2.0 * (double)features * (double)k * es / (double)splits;
            const int64_t groups = s.tiles_n * splits, more = groups % 256;
            const double us = base + (double)(groups / 256) * bytes * std::max(1 / rate, 256 / 5.5e6) +
                              (more > 0 ? bytes * std::max(1 / rate, (double)more / 5.5e6) : 0.0) +
                              (splits > 1 ? 4.0 + join * (double)splits : 0.0);
            if (best >= 0 && us >= best) continue;
            best = s.us = us;
            s.splits = splits;
        }
        // waves to share the columns: 2048 fill the chip
        const int most = s.shape == kFew16 ? 16 : 8;
        s.waves = 8;
        while (s.waves < most && s.waves * s.tiles_n * s.splits < 2048) s.waves *= 2;
        if (m <= 16) return s;
    }
    auto look = [&](const TileCost& c) {
        const int64_t tm = (m + c.rows - 1) / c.rows, tn = (n + c.cols - 1) / c.cols, tiles = tm * tn * outs;
        // more splits than make 2 rounds never pay
        const int64_t most = std::min((2 * c.slots + tiles - 1) / tiles, (steps + 3) / 4);
        for (int64_t splits = 1; splits <= std::max<int64_t>(most, 1); ++splits) {
            const int64_t per = (steps + splits - 1) / splits;
            if (splits > 1 && (steps + per - 1) / per != splits) continue;  // a split would be empty
            const double rounds = (double)((tiles * splits + c.slots - 1) / c.slots);
            const double us = rounds * (c.base + (tiles * splits <= 256 ? c.alone : c.step) * (double)per) +
                              (splits > 1 ? 4.0 + join * (double)splits : 0.0);
            if (best >= 0 && us >= best) continue;
            best = s.us = us;
            s.shape = c.shape;
            s.tiles_m = tm;
            s.tiles_n = tn;
            s.splits = splits;
            s.steps_per_split = per;
        }
    };
    const int64_t half = kind == kForward ? 2 : 1;  // a tile's columns are those of two weights
    if (short_rows(kind, m, n, k, es)) {
        look({kTileShort, 128, 128 / half, 512, 5, 2.0, 4.0});
        return s;
    }
    if (direct) {
        look(tile128(half, f32, true, false));
        look({kTile128Deep, 128, 128 / half, 256, 4, f32 ? 2.0 : 0.75, f32 ? 2.0 : 0.75});
        if (kind != kWeight) look({kTile64x128, 64, 128 / half, 512, 5, f32 ? 1.0 : 0.6, f32 ? 2.0 : 0.9});
        if (!f32) look({kTile256, 256, 256 / half, 256, 8, 1.7, 1.7});
        if (kind == kForward && !f32) look({kTile64, 64, 32, 256, 5, 0.48, 0.48});
        if (kind == kForward) look({kTile128x32, 128, 32, 256, 5, f32 ? 1.2 : 0.56, f32 ? 1.2 : 0.56});
    } else {
        look(tile128(half, f32, false, kind != kWeight));
        if (kind != kWeight) look({kTile64x128, 64, 128 / half, 768, 5, f32 ? 1.0 : 0.95, f32 ? 3.0 : 1.75});
        if (!f32) look({kTile256, 256, 256 / half, 256, 8, 2.1, 2.1});
    }
    if (f32) look({kTileSplit, 256, 128 / half, 256, 8, 2.3, 2.3});
    // (16 bits, aligned: a step takes as long as one of 64 x 128)
    if (kind == kInput && (f32 || !direct)) look({kTile32x128, 32, 128, 512, 5, f32 ? 0.7 : 0.6, f32 ? 1.1 : 0.9});
    return s;
}
int64_t product_workspace(const ProductShape& s, int64_t m, int64_t n, int outs) {
    return s.splits > 1 ? s.splits * outs * m * pitch_of(n) * 4 : 0;  // kForward: 2 outs
}
// Both gradients in one launch of tiles of 128: splits that give all workgroups
// about the same number of steps.  Taken where its time is below 0.9 of that of two
// launches, whose estimates are up to a fifth above what larger tiles take.  One
// launch and two, us (with the slopes): 2048 tokens x 1024 x 1024 bf16 35, 53; 512
// x 1001 x 1003 28, 44; 6 x 299 x 1855 17, 24; 1024 x 512 x 512 f32 39, 53; 1024 x
// 1536 x 4096 bf16 (0.92 of the estimate) 94, 84.
struct BothShape {
    ProductShape input, weight;
    double us;  // negative: not offered
};
BothShape both_shape(int64_t rows, int64_t cols, int64_t wide, int outs, int dtype, bool direct) {
    const bool f32 = dtype == PTORED_F32;
    const int es = esize_of(dtype);
    BothShape best{};
    best.us = -1;
    if (rows == 0 || cols == 0 || wide == 0 || outs == 0 || short_rows(kInput, rows, cols, wide, es) ||
        short_rows(kWeight, wide, cols, rows, es))
        return best;
    const int64_t depth = kStepBytes / es;
    const TileCost c = tile128(1, f32, direct, false);
    auto tiles = [](int64_t n) { return (n + 127) / 128; };
    const int64_t steps_in = (wide + depth - 1) / depth * 2, steps_w = (rows + depth - 1) / depth;
    const int64_t tiles_in = tiles(rows) * tiles(cols), tiles_w = tiles(wide) * tiles(cols) * outs;
    if (tiles_in + tiles_w > 4 * c.slots) return best;
    const int64_t most = std::max(steps_in, steps_w);
    for (int64_t target = 4;; target += std::max<int64_t>(1, target / 4)) {
        auto shape = [&](int64_t m, int64_t n, int64_t steps) {
            ProductShape s{};
            s.shape = kTile128;
            s.tiles_m = tiles(m);
            s.tiles_n = tiles(n);
            s.splits = (steps + target - 1) / target;
            s.steps_per_split = (steps + s.splits - 1) / s.splits;
            s.splits = (steps + s.steps_per_split - 1) / s.steps_per_split;
            return s;
        };
        const ProductShape in = shape(rows, cols, steps_in), w = shape(wide, cols, steps_w);
        const int64_t groups = tiles_in * in.splits + tiles_w * w.splits;
        const double longest = (double)std::max(in.steps_per_split, w.steps_per_split);
        const double share = (double)(tiles_in * steps_in + tiles_w * steps_w) / (double)c.slots;
        double us = groups <= 256 ? c.base + c.alone * longest
                                  : c.base * (double)((groups + c.slots - 1) / c.slots) +
                                        c.step * std::max(longest, share);
        const double sums = (in.splits > 1 ? (double)(in.splits * rows) : 0.0) +
                            (w.splits > 1 ? (double)(w.splits * outs * wide) : 0.0);
        if (sums > 0) us += 4.0 + sums * (double)cols * 8 / 4e6;
        if (best.us < 0 || us < best.us) best = {in, w, us};
        if (target >= most) break;
    }
    return best;
}
// (the input's partial sums begin where the weights' end)
int64_t both_workspace(const BothShape& b, int64_t rows, int64_t cols, int64_t wide, int outs) {
    return product_workspace(b.weight, wide, cols, outs) + product_workspace(b.input, rows, cols, 1);
}
bool launchable(const ProductShape& s, int outs) {
    return s.tiles_m <= kMaxTiles && s.tiles_n <= kMaxTiles &&
           s.tiles_m * s.tiles_n * outs * s.splits <= kMaxTiles;
}
void set_shape(ProductArgs& a, const ProductShape& s, bool direct) {
    a.tiles_m = (int32_t)s.tiles_m;
    a.tiles_n = (int32_t)s.tiles_n;
    a.splits = (int32_t)s.splits;
    a.steps_per_split = s.steps_per_split;
    a.shape = s.shape;
    a.waves = s.waves;
    a.direct = direct;
}
void set_a(ProductArgs& a, int i, const ptored_rows& r, int es) {
    a.a[i] = static_cast<const char*>(r.data);
    a.a_ld[i] = r.ld * es;
}
void set_b(ProductArgs& a, int i, const ptored_rows& r, int es) {
    a.b[i] = static_cast<const char*>(r.data);
    a.b_ld[i] = r.ld * es;
}

// ---------------------------------------------------------------- gradients

constexpr int64_t kInt = 0x7FFFFFFF;

bool grad_shape_ok(const ptored_grad& g, bool scaled) {
    if (!shape_ok(g.rows, g.cols)) return false;
    if (g.rows == 0 || g.cols == 0) return true;
    if (g.data == nullptr || (scaled && g.out == nullptr)) return false;
    return g.rows == 1 || (pitch_ok(g.rows, g.cols, g.ld) && (!scaled || pitch_ok(g.rows, g.cols, g.out_ld)));
}
bool grad_supported(const ptored_grad& g, bool scaled) {
    if (!float_type(g.dtype)) return false;
    if (scaled && g.out_dtype != PTORED_F32 && g.out_dtype != g.dtype) return false;
    if (g.rows == 0 || g.cols == 0) return true;
    // the table keeps a type beside the address
    if (reinterpret_cast<uintptr_t>(g.data) >> 48 != 0) return false;
    if (g.rows == 1) return g.cols < kGradMost;
    return g.rows <= kInt && g.ld <= kGradPitch && (!scaled || g.out_ld <= kGradPitch);
}
// Where the elements of a gradient that has some lie.
Extent lies(const ptored_grad& g, const void* p, int64_t ld, int dtype) {
    return extent_of(p, g.rows, g.cols, g.rows == 1 ? g.cols : ld, esize_of(dtype));
}
Extent data_of(const ptored_grad& g) { return lies(g, g.data, g.ld, g.dtype); }
Extent out_of(const ptored_grad& g) { return lies(g, g.out, g.out_ld, g.out_dtype); }

int64_t chunks_of(const ptored_grad& g) {
    return g.rows == 0 || g.cols == 0 ? 0 : grad_chunks(g.rows, g.cols, g.dtype);
}
int64_t all_chunks(const ptored_grad* grads, int64_t count) {
    int64_t n = 0;
    // (one of an unknown type is refused before its chunks matter)
    for (int64_t i = 0; i < count; ++i) n += chunks_of(grads[i]);
    return n;
}

// The workspace: the table of more gradients than a launch's arguments hold,
// then the partial sums.
int64_t grad_table_bytes(const ptored_grad* grads, int64_t count) {
    int64_t n = 0;
    for (int64_t i = 0; i < count; ++i) n += grads[i].rows > 0 && grads[i].cols > 0;
    return n > kGradEntries ? n * (int64_t)sizeof(GradEntry) : 0;
}

int64_t groups_of(int64_t chunks) { return std::min<int64_t>(chunks, kGradGroups); }

struct Span {
    Extent at;
    bool out;
};
// Whether an output among the gradients (or `more`, 2 spans) overlaps another
// buffer.  -1: no memory.
int grads_overlap(const ptored_grad* grads, int64_t count, const Span* more) {
    std::unique_ptr<Span[]> s(new (std::nothrow) Span[2 * (size_t)count + 2]);
    if (!s) return -1;
    size_t n = 0;
    for (int64_t i = 0; i < count; ++i) {
        const ptored_grad& g = grads[i];
        if (g.rows == 0 || g.cols == 0) continue;
        const bool same = g.data == g.out && g.dtype == g.out_dtype && (g.rows == 1 || g.ld == g.out_ld);
        s[n++] = {data_of(g), same};
        if (!same) s[n++] = {out_of(g), true};
    }
    for (int i = 0; i < 2; ++i)
        if (more[i].at.bytes > 0) s[n++] = more[i];
    std::sort(s.get(), s.get() + n, [](const Span& a, const Span& b) { return a.at.p < b.at.p; });
    uintptr_t any = 0, outs = 0;  // how far buffers, and outputs among them, reach so far
    bool apart = true;
    for (size_t i = 0; i < n && apart; ++i) {
        apart = s[i].at.p >= (s[i].out ? any : outs);
        const uintptr_t end = s[i].at.p + (uintptr_t)s[i].at.bytes;
        any = std::max(any, end);
        if (s[i].out) outs = std::max(outs, end);
    }
    // spans that meet, as column ranges of one matrix do: one by one
    for (size_t i = 0; i < n && !apart; ++i)
        for (size_t j = i + 1; j < n && s[j].at.p < s[i].at.p + (uintptr_t)s[i].at.bytes; ++j)
            if ((s[i].out || s[j].out) && meet(s[i].at, s[j].at)) return 1;
    return 0;
}

Span span(const void* p, int64_t bytes, bool out) { return {{reinterpret_cast<uintptr_t>(p), bytes, 0, bytes}, out}; }

// The checks of all three calls.  `sums`: the norm is taken.
int grads_checked(const ptored_grad* grads, int64_t count, bool scaled, bool sums, const float* norm,
                  const void* workspace, int64_t workspace_bytes) {
    if (count < 0 || count > kInt || (count > 0 && grads == nullptr) || norm == nullptr)
        return PTORED_ERR_INVALID_ARG;
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (!grad_shape_ok(grads[i], scaled)) return PTORED_ERR_INVALID_ARG;
        total += grads[i].rows * grads[i].cols;
        if (total > kMaxElems) return PTORED_ERR_INVALID_ARG;
    }
    for (int64_t i = 0; i < count; ++i)
        if (!grad_supported(grads[i], scaled)) return PTORED_ERR_UNSUPPORTED;
    const int64_t chunks = all_chunks(grads, count);
    if (chunks > kInt) return PTORED_ERR_UNSUPPORTED;
    const int64_t need = grad_table_bytes(grads, count) + (sums ? groups_of(chunks) * 8 : 0);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need ||
                     reinterpret_cast<uintptr_t>(workspace) % 16 != 0))
        return PTORED_ERR_INVALID_ARG;
    bool aligned = reinterpret_cast<uintptr_t>(norm) % 4 == 0;
    for (int64_t i = 0; i < count && aligned; ++i) {
        const ptored_grad& g = grads[i];
        if (g.rows == 0 || g.cols == 0) continue;
        aligned = reinterpret_cast<uintptr_t>(g.data) % (uintptr_t)esize_of(g.dtype) == 0 &&
                  (!scaled || reinterpret_cast<uintptr_t>(g.out) % (uintptr_t)esize_of(g.out_dtype) == 0);
    }
    if (!aligned) return PTORED_ERR_INVALID_ARG;
    const Span more[2] = {span(norm, 4, sums), span(workspace, need, true)};
    if (scaled) {
        const int over = grads_overlap(grads, count, more);
        return over < 0 ? PTORED_ERR_HIP : over > 0 ? PTORED_ERR_OVERLAP : PTORED_OK;
    }
    // only the norm and the workspace are written
    if (meet(more[0].at, more[1].at)) return PTORED_ERR_OVERLAP;
    for (int64_t i = 0; i < count; ++i) {
        if (grads[i].rows == 0 || grads[i].cols == 0) continue;
        for (const Span& m : more)
            if (meet(data_of(grads[i]), m.at)) return PTORED_ERR_OVERLAP;
    }
    return PTORED_OK;
}

// An entry's slots in a pack; 0 where they do not fit.
int packed(const ptored_grad& g, GradPack& p) {
    const int slots = g.rows == 1 ? 1 : 2, at = p.slots;
    if (at + slots > kGradSlots) return 0;
    const uint64_t type = (uint64_t)(g.dtype == g.out_dtype ? g.dtype : g.dtype + 3);
    p.heads[at / 32] |= 1u << at % 32;
    p.data[at] = reinterpret_cast<uint64_t>(g.data) | (uint64_t)(g.cols >> 32) << 48 | type << 56 |
                 (uint64_t)(slots - 1) << 59;
    p.out[at] = reinterpret_cast<uint64_t>(g.out);
    p.cols[at] = (uint32_t)g.cols;
    if (slots == 2) {
        p.data[at + 1] = (uint64_t)g.rows | (uint64_t)g.ld << 32;
        p.out[at + 1] = (uint64_t)g.out_ld;
        p.cols[at + 1] = 0;
    }
    p.slots += slots;
    return slots;
}

// The list of a call, in the arguments or put together in the workspace.
int list_of(const ptored_grad* grads, int64_t count, void* workspace, GradList& a, hipStream_t stream) {
    const int64_t bytes = grad_table_bytes(grads, count);
    GradPack p{};
    GradEntry* to = p.table = static_cast<GradEntry*>(workspace);
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        const ptored_grad& g = grads[i];
        if (g.rows == 0 || g.cols == 0) continue;
        if (bytes > 0) {
            if (packed(g, p) == 0) {
                const int rc = grad_table(p, stream);
                if (rc != kOk) return rc;
                p = GradPack{};
                p.table = to;
                p.first = (int32_t)chunks;
                packed(g, p);
            }
            ++to;
        } else {
            GradEntry& e = a.e[a.count];
            e.data = static_cast<const char*>(g.data);
            e.out = static_cast<char*>(g.out);
            e.cols = g.cols;
            e.rows = (int32_t)g.rows;
            e.ld = g.rows == 1 ? 0 : (int32_t)g.ld;
            e.out_ld = g.rows == 1 ? 0 : (int32_t)g.out_ld;
            e.first = (int32_t)chunks;
            e.type = g.dtype | g.out_dtype << 8;
        }
        ++a.count;
        chunks += chunks_of(g);
    }
    if (bytes > 0) {
        const int rc = grad_table(p, stream);
        if (rc != kOk) return rc;
        a.table = static_cast<const GradEntry*>(workspace);
    }
    a.chunks = (int32_t)chunks;
    a.groups = (int32_t)groups_of(chunks);
    a.sums = reinterpret_cast<double*>(static_cast<char*>(workspace) + bytes);
    return kOk;
}

// The list and its partial sums.
int run_sums(const ptored_grad* grads, int64_t count, void* workspace, GradList& a,
             hipStream_t stream) {
    int rc = list_of(grads, count, workspace, a, stream);
    if (rc == kOk && a.groups > 0) rc = grad_sums(a, stream);
    a.all = a.sums;
    a.all_count = a.groups;
    return rc;
}

}  // namespace
}  // namespace step
}  // namespace ptored

using namespace ptored::step;
using ptored::block::Buffers;
using ptored::block::esize_of;
using ptored::block::float_type;
using ptored::block::mat;
using ptored::block::shape_ok;
using ptored::block::status_of;

extern "C" int ptored_layer_norm(const void* const* parts, int nranks, int64_t part_ld,
                                 const ptored_layer_norm_params* params, ptored_rows x,
                                 ptored_rows x_out, ptored_rows z, float* mean, float* rstd,
                                 hipStream_t stream) {
    if (nranks < 0 || nranks > PTORED_MAX_RANKS || (nranks > 0 && parts == nullptr))
        return PTORED_ERR_INVALID_ARG;
    if (!layer_valid(params) || x.data == nullptr || !(params->eps >= 0.0f))
        return PTORED_ERR_INVALID_ARG;
    const ptored_layer_norm_params& p = *params;
    const int es = esize_of(p.dtype), ws = esize_of(p.weight_dtype);
    Buffers b;
    bool ok = b.rows(x.data, p.rows, p.cols, x.ld, es, false);
    for (int r = 0; r < nranks && ok; ++r)
        ok = parts[r] != nullptr && b.rows(parts[r], p.rows, p.cols, part_ld, es, false);
    ok = ok && b.rows(x_out.data, p.rows, p.cols, x_out.ld, es, true) &&
         b.rows(z.data, p.rows, p.cols, z.ld, es, true);
    if (!ok) return PTORED_ERR_INVALID_ARG;
    if (!layer_supported(p)) return PTORED_ERR_UNSUPPORTED;
    b.vec(p.weight, p.cols * ws, ws, false);
    b.vec(p.bias, p.cols * ws, ws, false);
    b.vec(mean, p.rows * 4, 4, true);
    b.vec(rstd, p.rows * 4, 4, true);
    if (!b.aligned()) return PTORED_ERR_INVALID_ARG;
    if (!b.disjoint()) return PTORED_ERR_OVERLAP;
    if (p.rows == 0 || p.cols == 0) return PTORED_OK;

    LayerNormArgs a{};
    for (int r = 0; r < nranks; ++r) a.part[r] = static_cast<const char*>(parts[r]);
    a.part_ld = part_ld * es;
    a.nranks = nranks;
    a.rows = p.rows;
    a.cols = (int32_t)p.cols;
    a.x = mat(x, es);
    a.x_out = mat(x_out, es);
    a.z = mat(z, es);
    a.w = static_cast<const char*>(p.weight);
    a.b = static_cast<const char*>(p.bias);
    a.mean = mean;
    a.rstd = rstd;
    a.w_f32 = p.weight_dtype == PTORED_F32;
    a.eps = p.eps;
    a.inv_cols = 1.0f / (float)p.cols;
    return status_of(PTORED_BY_TYPE(layer_norm, p.dtype, a, stream));
}

extern "C" int ptored_layer_norm_backward_workspace(int64_t rows, int64_t cols, int64_t* bytes) {
    if (bytes == nullptr || !shape_ok(rows, cols)) return PTORED_ERR_INVALID_ARG;
    if (cols > PTORED_BLOCK_MAX_COLS) return PTORED_ERR_UNSUPPORTED;
    // of any type
    *bytes = layer_workspace(std::max(layer_chunks(rows, cols, PTORED_F32),
                                      layer_chunks(rows, cols, PTORED_BF16)), cols);
    return PTORED_OK;
}

extern "C" int ptored_layer_norm_backward(const ptored_layer_norm_params* params, ptored_rows dz,
                                          ptored_rows dx_out, ptored_rows x_out, const float* mean,
                                          const float* rstd, ptored_rows dx, void* dweight,
                                          void* dbias, void* workspace, int64_t workspace_bytes,
                                          hipStream_t stream) {
    if (!layer_valid(params) || dz.data == nullptr || x_out.data == nullptr || mean == nullptr ||
        rstd == nullptr)
        return PTORED_ERR_INVALID_ARG;
    const ptored_layer_norm_params& p = *params;
    const int es = esize_of(p.dtype), ws = esize_of(p.weight_dtype);
    Buffers b;
    if (!b.rows(dz.data, p.rows, p.cols, dz.ld, es, false) ||
        !b.rows(dx_out.data, p.rows, p.cols, dx_out.ld, es, false) ||
        !b.rows(x_out.data, p.rows, p.cols, x_out.ld, es, false) ||
        !b.rows(dx.data, p.rows, p.cols, dx.ld, es, true))
        return PTORED_ERR_INVALID_ARG;
    if (!layer_supported(p)) return PTORED_ERR_UNSUPPORTED;
    b.vec(p.weight, p.cols * ws, ws, false);
    b.vec(mean, p.rows * 4, 4, false);
    b.vec(rstd, p.rows * 4, 4, false);
    b.vec(dweight, p.cols * ws, ws, true);
    b.vec(dbias, p.cols * ws, ws, true);
    const bool sums = dweight != nullptr || dbias != nullptr;
    const int64_t chunks = layer_chunks(p.rows, p.cols, p.dtype);
    const int64_t need = sums ? layer_workspace(chunks, p.cols) : 0;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return PTORED_ERR_INVALID_ARG;
    if (need > 0) b.vec(workspace, need, 16, true);
    if (!b.aligned()) return PTORED_ERR_INVALID_ARG;
    if (!b.disjoint()) return PTORED_ERR_OVERLAP;
    if (p.cols == 0 || (dx.data == nullptr && !sums)) return PTORED_OK;

    LayerGradArgs a{};
    a.rows = p.rows;
    a.cols = (int32_t)p.cols;
    a.dz = mat(dz, es);
    a.dxo = mat(dx_out, es);
    a.x = mat(x_out, es);
    a.dx = mat(dx, es);
    a.w = static_cast<const char*>(p.weight);
    a.mean = mean;
    a.rstd = rstd;
    a.ws = sums ? static_cast<float*>(workspace) : nullptr;
    a.dw = static_cast<char*>(dweight);
    a.db = static_cast<char*>(dbias);
    a.chunks = chunks;
    a.ws_pitch = pitch_of(p.cols);
    a.w_f32 = p.weight_dtype == PTORED_F32;
    a.inv_cols = 1.0f / (float)p.cols;
    return status_of(PTORED_BY_TYPE(layer_grad, p.dtype, a, stream));
}

extern "C" int ptored_gated_ffn(const ptored_ffn_params* params, ptored_rows x, ptored_rows w_gate,
                                ptored_rows w_up, ptored_rows y, ptored_rows gate, ptored_rows up,
                                void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!ffn_valid(params) || x.data == nullptr || w_gate.data == nullptr || w_up.data == nullptr ||
        y.data == nullptr)
        return PTORED_ERR_INVALID_ARG;
    const ptored_ffn_params& p = *params;
    const int es = esize_of(p.dtype);
    Buffers b;
    if (!b.rows(x.data, p.rows, p.cols, x.ld, es, false, false) ||
        !b.rows(w_gate.data, p.wide, p.cols, w_gate.ld, es, false, false) ||
        !b.rows(w_up.data, p.wide, p.cols, w_up.ld, es, false, false) ||
        !b.rows(y.data, p.rows, p.wide, y.ld, es, true, false) ||
        !b.rows(gate.data, p.rows, p.wide, gate.ld, es, true, false) ||
        !b.rows(up.data, p.rows, p.wide, up.ld, es, true, false))
        return PTORED_ERR_INVALID_ARG;
    if (!ffn_supported(p) || !widths_supported(p, es) || !pitch_supported(x, p.rows, es) ||
        !pitch_supported(w_gate, p.wide, es) || !pitch_supported(w_up, p.wide, es))
        return PTORED_ERR_UNSUPPORTED;
    const bool direct = direct_of(x, p.rows, p.cols, es) && direct_of(w_gate, p.wide, p.cols, es) &&
                        direct_of(w_up, p.wide, p.cols, es);
    const ProductShape s = product_shape(kForward, p.rows, p.wide, p.cols, 1, p.dtype, direct);
    if (!launchable(s, 1)) return PTORED_ERR_UNSUPPORTED;
    const int64_t need = product_workspace(s, p.rows, p.wide, 2);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return PTORED_ERR_INVALID_ARG;
    if (need > 0) b.vec(workspace, need, 16, true);
    if (!b.aligned()) return PTORED_ERR_INVALID_ARG;
    if (!b.disjoint()) return PTORED_ERR_OVERLAP;
    if (p.rows == 0 || p.wide == 0) return PTORED_OK;

    ProductArgs a{};
    set_a(a, 0, operand(x, p.rows, p.cols), es);
    set_b(a, 0, operand(w_gate, p.wide, p.cols), es);
    set_b(a, 1, operand(w_up, p.wide, p.cols), es);
    a.m = p.rows;
    a.n = p.wide;
    a.k = p.cols;
    a.out[0] = mat(y, es);
    a.gate = mat(gate, es);
    a.up = mat(up, es);
    a.outs = 1;
    a.activation = p.activation;
    a.ws = static_cast<float*>(workspace);
    a.ws_ld = pitch_of(p.wide);
    set_shape(a, s, direct);
    return status_of(PTORED_BY_TYPE(product_forward, p.dtype, a, stream));
}

extern "C" int ptored_gated_ffn_workspace(int64_t rows, int64_t cols, int64_t wide, int dtype,
                                          int64_t* bytes) {
    if (bytes == nullptr || !shape_ok(rows, cols) || !shape_ok(rows, wide) || !shape_ok(wide, cols))
        return PTORED_ERR_INVALID_ARG;
    if (!float_type(dtype)) return PTORED_ERR_UNSUPPORTED;
    *bytes = 0;  // of any alignment
    for (const bool direct : {false, true})
        *bytes = std::max(*bytes, product_workspace(product_shape(kForward, rows, wide, cols, 1, dtype, direct),
                                                    rows, wide, 2));
    return PTORED_OK;
}

extern "C" int ptored_gated_ffn_backward_workspace(int64_t rows, int64_t cols, int64_t wide,
                                                   int dtype, int64_t* bytes) {
    if (bytes == nullptr || !shape_ok(rows, cols) || !shape_ok(rows, wide) || !shape_ok(wide, cols))
        return PTORED_ERR_INVALID_ARG;
    if (!float_type(dtype)) return PTORED_ERR_UNSUPPORTED;
    int64_t most = 0;  // of any alignment and any choice of gradients; products take turns, or both are one launch
    for (const bool direct : {false, true}) {
        most = std::max(most, product_workspace(product_shape(kInput, rows, cols, wide, 1, dtype, direct),
                                                rows, cols, 1));
        for (const int outs : {1, 2}) {
            most = std::max(most, product_workspace(product_shape(kWeight, wide, cols, rows, outs, dtype,
                                                                  direct), wide, cols, outs));
            const BothShape both = both_shape(rows, cols, wide, outs, dtype, direct);
            if (both.us >= 0) most = std::max(most, both_workspace(both, rows, cols, wide, outs));
        }
    }
    *bytes = most;
    return PTORED_OK;
}

extern "C" int ptored_gated_ffn_backward(const ptored_ffn_params* params,
                                         const ptored_ffn_grad_io* io, hipStream_t stream) {
    if (!ffn_valid(params) || io == nullptr || io->dy.data == nullptr || io->gate.data == nullptr ||
        io->up.data == nullptr || io->dgate.data == nullptr || io->dup.data == nullptr)
        return PTORED_ERR_INVALID_ARG;
    const ptored_ffn_params& p = *params;
    const bool input = io->dx.data != nullptr;
    const int outs = (io->dw_gate.data != nullptr) + (io->dw_up.data != nullptr);
    if ((outs > 0 && io->x.data == nullptr) ||
        (input && (io->w_gate.data == nullptr || io->w_up.data == nullptr)))
        return PTORED_ERR_INVALID_ARG;
    const int es = esize_of(p.dtype), ws = esize_of(io->dw_dtype);
    // what no product reads is not looked at
    const ptored_rows none{nullptr, 0};
    const ptored_rows x = outs > 0 ? io->x : none;
    const ptored_rows wg = input ? io->w_gate : none, wu = input ? io->w_up : none;
    Buffers b;
    if (!b.rows(io->dy.data, p.rows, p.wide, io->dy.ld, es, false) ||
        !b.rows(io->gate.data, p.rows, p.wide, io->gate.ld, es, false) ||
        !b.rows(io->up.data, p.rows, p.wide, io->up.ld, es, false) ||
        !b.rows(io->dgate.data, p.rows, p.wide, io->dgate.ld, es, true) ||
        !b.rows(io->dup.data, p.rows, p.wide, io->dup.ld, es, true) ||
        !b.rows(x.data, p.rows, p.cols, x.ld, es, false, false) ||
        !b.rows(wg.data, p.wide, p.cols, wg.ld, es, false, false) ||
        !b.rows(wu.data, p.wide, p.cols, wu.ld, es, false, false) ||
        !b.rows(io->dx.data, p.rows, p.cols, io->dx.ld, es, true, false) ||
        !b.rows(io->dw_gate.data, p.wide, p.cols, io->dw_gate.ld, ws, true, false) ||
        !b.rows(io->dw_up.data, p.wide, p.cols, io->dw_up.ld, ws, true, false))
        return PTORED_ERR_INVALID_ARG;
    if (!ffn_supported(p) || (outs > 0 && io->dw_dtype != PTORED_F32 && io->dw_dtype != p.dtype))
        return PTORED_ERR_UNSUPPORTED;
    // what a product reads; the slopes alone have no limits
    if ((input || outs > 0) &&
        (!widths_supported(p, es) || !pitch_supported(io->dgate, p.rows, es) || !pitch_supported(io->dup, p.rows, es) ||
         !pitch_supported(x, p.rows, es) || !pitch_supported(wg, p.wide, es) || !pitch_supported(wu, p.wide, es)))
        return PTORED_ERR_UNSUPPORTED;
    const bool whole = direct_of(io->dgate, p.rows, p.wide, es) && direct_of(io->dup, p.rows, p.wide, es);
    const bool direct_in = whole && direct_of(wg, p.wide, p.cols, es) && direct_of(wu, p.wide, p.cols, es);
    const bool direct_w = whole && direct_of(x, p.rows, p.cols, es);
    const ProductShape si =
        input ? product_shape(kInput, p.rows, p.cols, p.wide, 1, p.dtype, direct_in) : ProductShape{};
    const ProductShape sw =
        outs > 0 ? product_shape(kWeight, p.wide, p.cols, p.rows, outs, p.dtype, direct_w) : ProductShape{};
    if ((input && !launchable(si, 1)) || (outs > 0 && !launchable(sw, outs)))
        return PTORED_ERR_UNSUPPORTED;
    const bool direct_both = direct_in && direct_w;
    const BothShape sb = input && outs > 0 ? both_shape(p.rows, p.cols, p.wide, outs, p.dtype, direct_both)
                                           : BothShape{{}, {}, -1};
    const bool both = sb.us >= 0 && sb.us < 0.9 * (si.us + sw.us);
    const int64_t need = both ? both_workspace(sb, p.rows, p.cols, p.wide, outs)
                              : std::max(input ? product_workspace(si, p.rows, p.cols, 1) : 0,
                                         outs > 0 ? product_workspace(sw, p.wide, p.cols, outs) : 0);
    if (need > 0 && (io->workspace == nullptr || io->workspace_bytes < need))
        return PTORED_ERR_INVALID_ARG;
    if (need > 0) b.vec(io->workspace, need, 16, true);
    if (!b.aligned()) return PTORED_ERR_INVALID_ARG;
    if (!b.disjoint()) return PTORED_ERR_OVERLAP;

    if (p.rows > 0 && p.wide > 0) {
        const SlopeArgs a{mat(io->dy, es), mat(io->gate, es), mat(io->up, es), mat(io->dgate, es),
                          mat(io->dup, es), p.rows, p.wide, p.activation};
        const int rc = PTORED_BY_TYPE(product_slope, p.dtype, a, stream);
        if (rc != ptored::block::kOk) return status_of(rc);
    }
    ProductPair pair{};
    if (input && p.rows > 0 && p.cols > 0) {
        ProductArgs& a = pair.input;
        set_a(a, 0, operand(io->dgate, p.rows, p.wide), es);
        set_a(a, 1, operand(io->dup, p.rows, p.wide), es);
        set_b(a, 0, operand(wg, p.wide, p.cols), es);
        set_b(a, 1, operand(wu, p.wide, p.cols), es);
        a.m = p.rows;
        a.n = p.cols;
        a.k = p.wide;
        a.out[0] = mat(io->dx, es);
        a.outs = 1;
        a.out_f32 = p.dtype == PTORED_F32;
        a.ws = static_cast<float*>(io->workspace);
        a.ws_ld = pitch_of(p.cols);
        if (both) a.ws += product_workspace(sb.weight, p.wide, p.cols, outs) / 4;
        set_shape(a, both ? sb.input : si, both ? direct_both : direct_in);
    }
    if (input && !both && p.rows > 0 && p.cols > 0) {
        const int rc = PTORED_BY_TYPE(product_input, p.dtype, pair.input, stream);
        if (rc != ptored::block::kOk) return status_of(rc);
    }
    if (outs > 0 && p.wide > 0 && p.cols > 0 && !(p.rows == 0 && io->accumulate)) {
        ProductArgs& a = pair.weight;
        int n = 0;
        for (int i = 0; i < 2; ++i) {
            const ptored_rows& dw = i == 0 ? io->dw_gate : io->dw_up;
            if (dw.data == nullptr) continue;
            set_a(a, n, operand(i == 0 ? io->dgate : io->dup, p.rows, p.wide), es);
            a.out[n++] = mat(dw, ws);
        }
        set_b(a, 0, operand(x, p.rows, p.cols), es);
        a.m = p.wide;
        a.n = p.cols;
        a.k = p.rows;
        a.outs = outs;
        a.out_f32 = io->dw_dtype == PTORED_F32;
        a.accumulate = io->accumulate != 0;
        a.ws = static_cast<float*>(io->workspace);
        a.ws_ld = pitch_of(p.cols);
        set_shape(a, both ? sb.weight : sw, both ? direct_both : direct_w);
        pair.first = a.tiles_m * a.tiles_n * a.outs * a.splits;
        const int rc = both ? PTORED_BY_TYPE(product_both, p.dtype, pair, stream)
                            : PTORED_BY_TYPE(product_weight, p.dtype, a, stream);
        if (rc != ptored::block::kOk) return status_of(rc);
    }
    return PTORED_OK;
}

extern "C" int ptored_grad_norm_workspace(const ptored_grad* grads, int64_t count, int64_t* bytes) {
    if (bytes == nullptr || count < 0 || (count > 0 && grads == nullptr)) return PTORED_ERR_INVALID_ARG;
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (!shape_ok(grads[i].rows, grads[i].cols)) return PTORED_ERR_INVALID_ARG;
        if (!float_type(grads[i].dtype)) return PTORED_ERR_UNSUPPORTED;
        total += grads[i].rows * grads[i].cols;
        if (total > ptored::block::kMaxElems) return PTORED_ERR_INVALID_ARG;
    }
    *bytes = grad_table_bytes(grads, count) + groups_of(all_chunks(grads, count)) * 8;
    return PTORED_OK;
}

extern "C" int ptored_grad_norm(const ptored_grad* grads, int64_t count, float* norm, void* workspace,
                                int64_t workspace_bytes, hipStream_t stream) {
    const int st = grads_checked(grads, count, false, true, norm, workspace, workspace_bytes);
    if (st != PTORED_OK) return st;
    GradList a{};
    const int rc = run_sums(grads, count, workspace, a, stream);
    if (rc != ptored::block::kOk) return status_of(rc);
    a.norm = norm;
    return status_of(grad_join(a, stream));
}

extern "C" int ptored_grad_scale(const ptored_grad* grads, int64_t count, const float* norm,
                                 float max_norm, void* workspace, int64_t workspace_bytes,
                                 hipStream_t stream) {
    if (!(max_norm >= 0.0f)) return PTORED_ERR_INVALID_ARG;
    const int st = grads_checked(grads, count, true, false, norm, workspace, workspace_bytes);
    if (st != PTORED_OK) return st;
    GradList a{};
    const int rc = list_of(grads, count, workspace, a, stream);
    if (rc != ptored::block::kOk || a.groups == 0) return status_of(rc);
    a.norm = const_cast<float*>(norm);  // read only: no sums are given
    a.max_norm = max_norm;
    return status_of(grad_scale(a, stream));
}

extern "C" int ptored_grad_clip(const ptored_grad* grads, int64_t count, float max_norm, float* norm,
                                void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    if (!(max_norm >= 0.0f)) return PTORED_ERR_INVALID_ARG;
    const int st = grads_checked(grads, count, true, true, norm, workspace, workspace_bytes);
    if (st != PTORED_OK) return st;
    GradList a{};
    const int rc = run_sums(grads, count, workspace, a, stream);
    if (rc != ptored::block::kOk) return status_of(rc);
    a.norm = norm;
    a.max_norm = max_norm;
    return status_of(a.groups > 0 ? grad_scale(a, stream) : grad_join(a, stream));
}
