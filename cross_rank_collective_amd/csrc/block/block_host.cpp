// block_host.cpp -- C ABI of the block-boundary operators and of the 8-bit
// activation checkpoints: argument checks, work splits, launches.
//
// Every argument check runs before the first HIP call, so every error status
// is reachable without a GPU.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "block_plan.h"

namespace ptored {
namespace block {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 60;
constexpr int64_t kMaxCols = int64_t(1) << 30;

int esize_of(int dtype) { return dtype == PTORED_F32 ? 4 : 2; }
bool float_type(int dtype) { return dtype >= PTORED_F32 && dtype <= PTORED_F16; }

bool shape_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && cols >= 0 && (cols == 0 || rows <= kMaxElems / cols);
}
// A pitch that holds the columns and whose byte extent fits.
bool pitch_ok(int64_t rows, int64_t cols, int64_t ld) {
    return ld >= cols && (ld == 0 || rows <= kMaxElems / ld);
}
int64_t blocks_of(int64_t cols) {
    return (cols + PTORED_CHECKPOINT_BLOCK - 1) / PTORED_CHECKPOINT_BLOCK;
}

// The buffers of a call: checks each one's shape, alignment and overlaps.
class Buffers {
  public:
    // A matrix that the call reads (`out` false) or writes; absent if null.
    // `whole`: T x D, each row read and written by one workgroup alone.
    bool rows(const void* p, int64_t n, int64_t cols, int64_t ld, int es, bool out,
              bool whole = true) {
        if (p == nullptr) return true;
        if (!pitch_ok(n, cols, ld)) return false;
        // a single row has no pitch of its own
        add(p, n > 0 && cols > 0 ? ((n - 1) * ld + cols) * es : 0, (n > 1 ? ld : cols) * es, es, out,
            whole);
        return true;
    }
    bool kept(const ptored_checkpoint& k, int64_t n, int64_t cols, bool out) {
        if (k.q == nullptr) return true;
        if (k.scales == nullptr) return false;
        const int64_t nb = blocks_of(cols);
        if (!pitch_ok(n, cols, k.q_ld) || !pitch_ok(n, nb, k.scales_ld)) return false;
        const bool any = n > 0 && cols > 0;
        add(k.q, any ? (n - 1) * k.q_ld + cols : 0, k.q_ld, 1, out, false);
        add(k.scales, any ? (n - 1) * k.scales_ld + nb : 0, k.scales_ld, 1, out, false);
        return true;
    }
    void vec(const void* p, int64_t bytes, int align, bool out) {
        if (p != nullptr) add(p, bytes, 0, align, out, false);
    }
    bool aligned() const {
        for (int i = 0; i < n_; ++i)
            if (b_[i].p % (uintptr_t)b_[i].align != 0) return false;
        return true;
    }
    // No output overlaps another buffer, but for one that is exactly an input
    // matrix (gates and their gradients apart): same address, pitch and element size.
    bool disjoint() const {
        for (int i = 0; i < n_; ++i) {
            if (!b_[i].out || b_[i].bytes == 0) continue;
            for (int j = 0; j < n_; ++j) {
                if (i == j || b_[j].bytes == 0) continue;
                const Buf &o = b_[i], &x = b_[j];
                if (o.p >= x.p + (uintptr_t)x.bytes || x.p >= o.p + (uintptr_t)o.bytes) continue;
                const bool same = !x.out && o.matrix && x.matrix && o.p == x.p &&
                                  o.pitch == x.pitch && o.align == x.align;
                if (!same) return false;
            }
        }
        return true;
    }

  private:
    struct Buf {
        uintptr_t p;
        int64_t bytes, pitch;
        int align;
        bool out, matrix;
    };
    void add(const void* p, int64_t bytes, int64_t pitch, int align, bool out, bool matrix) {
        b_[n_++] = {reinterpret_cast<uintptr_t>(p), bytes, pitch, align, out, matrix};
    }
    Buf b_[PTORED_MAX_RANKS + 24];
    int n_ = 0;
};

Mat mat(const ptored_rows& r, int es) { return {static_cast<char*>(r.data), r.ld * es}; }
Kept kept(const ptored_checkpoint& k) {
    return {static_cast<int8_t*>(k.q), k.q_ld, static_cast<uint8_t*>(k.scales), k.scales_ld};
}

// The checks that both passes share, in two parts: counts and pointers, then
// types and limits.
bool params_valid(const ptored_block_params* p) {
    if (p == nullptr || !shape_ok(p->rows, p->cols)) return false;
    if (p->gate.data == nullptr) return true;
    return p->gate_rows > 0 && p->rows % p->gate_rows == 0;
}
bool params_supported(const ptored_block_params* p) {
    return float_type(p->dtype) && (p->weight_dtype == PTORED_F32 || p->weight_dtype == p->dtype) &&
           p->cols <= PTORED_BLOCK_MAX_COLS;
}

int status_of(int rc) { return rc == kOk ? PTORED_OK : PTORED_ERR_HIP; }

#define PTORED_BY_TYPE(f, dtype, ...)                            \
    ((dtype) == PTORED_F32    ? f##_f32(__VA_ARGS__)             \
     : (dtype) == PTORED_BF16 ? f##_bf16(__VA_ARGS__)            \
                              : f##_f16(__VA_ARGS__))

// The backward pass cuts the rows into as many chunks as there are workgroups
// at once on the chip: with fewer, compute units idle; with more, the last
// ones run alone and the partial rows that chunks leave (8 bytes a column,
// written and read) grow.  A wave is 64 slots wide; its registers leave room
// for 16 waves of 8-element slots on a compute unit and for 20 of 4.  But with
// work for all compute units the rows are not cut below chunks of 5: with fewer
// the partial rows weigh as much as the rows' own data (both kernels, bf16,
// packed: 4096 x 1024 28 us without the rule, 24 with 3 rows, 21 with 5, 22 with
// 7; 1511 x 2520 27, 23, 23, 22; 512 x 4096 22, 17 with 2 rows).  Where a gate
// row is a little longer than that, its equal parts are shorter (6 rows: 3 and 3).
GradSplit grad_split(int64_t rows, int64_t cols, int64_t gate_rows, int dtype,
                     bool in_order = false) {
    GradSplit s{};
    if (rows == 0 || cols == 0) return s;
    const int64_t slot = dtype == PTORED_F32 ? 4 : 8, room = dtype == PTORED_F32 ? 20 : 16;
    const int64_t waves = std::min<int64_t>(16, (cols + 64 * slot - 1) / (64 * slot));
    const int64_t target = 256 * (room / waves);
    const int64_t per = std::max((rows + target - 1) / target,
                                 std::min<int64_t>(5, (rows + 255) / 256));
    const int64_t unit = gate_rows > 0 ? rows / gate_rows : rows;
    if (gate_rows > 0 && unit <= per) {  // whole gate rows inside a chunk
        s.unit_rows = rows;
        s.chunk_rows = per / unit * unit;
        s.chunks_per_unit = (rows + s.chunk_rows - 1) / s.chunk_rows;
        s.chunks = s.chunks_per_unit;
        s.chunk_first = unit == 1 ? 1 : s.chunk_rows;
        s.row_step = unit == 1 ? s.chunks : 1;
        s.gate_direct = 1;
        return s;
    }
    s.unit_rows = unit;
    s.chunks_per_unit = (unit + per - 1) / per;
    s.chunk_rows = (unit + s.chunks_per_unit - 1) / s.chunks_per_unit;
    s.chunks = rows / unit * s.chunks_per_unit;
    s.chunk_first = in_order ? s.chunk_rows : 1;
    s.row_step = in_order ? 1 : s.chunks_per_unit;
    return s;
}

// Columns of a partial row: whole vectors of 4.
int64_t grad_pitch(int64_t cols) { return (cols + 3) / 4 * 4; }

int64_t grad_workspace(int64_t cols, int64_t gate_rows, const GradSplit& s) {
    return s.chunks * grad_pitch(cols) * 4 * (gate_rows > 0 && !s.gate_direct ? 3 : 2);
}

struct WgradShape {
    int64_t tiles_m, tiles_n, splits, rows_per_split;
    int shape;
};

// Tiles and splits of the weight gradient, by estimated time.  A tile of
// `tokens` takes about base + step tokens / 64 us, one tile at a time on each
// of 256 compute units (the figures are fits to sizes from 64 to 32768 tokens
// and 128 to 4096 columns).  Splitting the tokens shortens a tile's walk and
// fills idle compute units; each split writes its partial dw, which is read
// again by a second kernel: 4 us and the bytes at 2.6 TB/s.  So with few
// tiles the best number of splits is near sqrt(walk / time of one dw), as
// long as the tiles of all splits still run at once.
// Measured, us, best splits of 128 x 128 tiles against 256 x 256, bf16: 1024
// tokens x 2048 x 2048 19 / 39, 4096 x 2048 x 2048 48 / 57, 16384 x 4096 x 512 91
// / 83, 8192 x 4096 x 4096 343 / 244; f16: 20 / 43, 50 / 62, 96 / 90, 369 / 280
// (its kernel of 256 x 256 spills registers and still wins where tiles are many).
// 32768 x 640 x 512 with 1, 6, 12 and 25 splits 267, 60, 41 and 49.
struct WgradCost {
    int shape;
    int64_t tm, tn;
    double base, step;
};
constexpr int64_t kTokens = 128;  // rows of a split: a multiple of two steps

double wgrad_time(const WgradCost& c, int64_t rows, int64_t tiles, int64_t splits, double dw_us) {
    const int64_t per = (rows + splits - 1) / splits;
    const int64_t rounds = (tiles * splits + 255) / 256;
    return (double)rounds * (c.base + c.step * (double)per / 64) +
           (splits > 1 ? 4.0 + dw_us * (double)splits : 0.0);
}

WgradShape wgrad_shape(int64_t rows, int64_t outs, int64_t cols, int dtype) {
    static constexpr WgradCost k16[] = {{kWgradTile, 128, 128, 8.0, 0.7},
                                        {kWgradWide, 256, 256, 17.0, 1.8}};
    static constexpr WgradCost k32[] = {{kWgradTile, 128, 256, 14.0, 2.4}};
    static constexpr WgradCost kFew[] = {{kWgradFew, 128, 128, 10.0, 1.0}};
    WgradShape w{};
    if (outs == 0 || cols == 0) return w;
    const bool few = outs < 8 || cols < 16;
    const WgradCost* costs = few ? kFew : dtype == PTORED_F32 ? k32 : k16;
    const int count = !few && dtype != PTORED_F32 ? 2 : 1;
    const double dw_us = (double)outs * (double)cols * 4 / 2.6e6;
    double best = -1;
    for (int i = 0; i < count; ++i) {
        const WgradCost& c = costs[i];
        const int64_t tm = (outs + c.tm - 1) / c.tm, tn = (cols + c.tn - 1) / c.tn, tiles = tm * tn;
        int64_t splits = 1;
        if (rows > kTokens && tiles <= 128) {
            const int64_t room = std::min(256 / tiles, (rows + kTokens - 1) / kTokens);
            const double ideal = std::sqrt(c.step * (double)rows / 64 / dw_us);
            const int64_t s = ideal < (double)room ? std::max<int64_t>(1, (int64_t)(ideal + 0.5)) : room;
            if (wgrad_time(c, rows, tiles, s, dw_us) < wgrad_time(c, rows, tiles, 1, dw_us))
                splits = s;
        }
        const double us = wgrad_time(c, rows, tiles, splits, dw_us);
        if (best >= 0 && us >= best) continue;
        best = us;
        w.shape = c.shape;
        w.tiles_m = tm;
        w.tiles_n = tn;
        w.splits = splits;
    }
    if (rows == 0) {
        w.splits = 0;
        return w;
    }
    const int64_t per = ((rows + w.splits - 1) / w.splits + kTokens - 1) / kTokens * kTokens;
    w.rows_per_split = per;
    w.splits = (rows + per - 1) / per;
    return w;
}

// Columns of a partial row: whole vectors of 4.
int64_t wgrad_pitch(int64_t cols) { return (cols + 3) / 4 * 4; }

int64_t wgrad_workspace(int64_t outs, int64_t cols, const WgradShape& w) {
    return w.splits > 1 ? w.splits * outs * wgrad_pitch(cols) * 4 : 0;
}

int checkpoint_args(const ptored_rows& x, int64_t rows, int64_t cols, int dtype,
                    const ptored_checkpoint& k, bool packs) {
    if (x.data == nullptr || k.q == nullptr || k.scales == nullptr) return PTORED_ERR_INVALID_ARG;
    Buffers b;
    if (!shape_ok(rows, cols) || cols > kMaxCols ||
        !b.rows(x.data, rows, cols, x.ld, esize_of(dtype), !packs) ||
        !b.kept(k, rows, cols, packs))
        return PTORED_ERR_INVALID_ARG;
    if (!float_type(dtype)) return PTORED_ERR_UNSUPPORTED;
    if (!b.aligned()) return PTORED_ERR_INVALID_ARG;
    return b.disjoint() ? PTORED_OK : PTORED_ERR_OVERLAP;
}

}  // namespace
}  // namespace block
}  // namespace ptored

using namespace ptored::block;

extern "C" int ptored_block_norm(const void* const* parts, int nranks, int64_t part_ld,
                                 const ptored_block_params* params, const ptored_block_io* io,
                                 hipStream_t stream) {
    if (nranks < 0 || nranks > PTORED_MAX_RANKS || (nranks > 0 && parts == nullptr))
        return PTORED_ERR_INVALID_ARG;
    if (!params_valid(params) || io == nullptr || io->x.data == nullptr)
        return PTORED_ERR_INVALID_ARG;
    const ptored_block_params& p = *params;
    if (!(p.eps >= 0.0f)) return PTORED_ERR_INVALID_ARG;
    if (nranks == 0 && (p.post_weight || p.gate.data || io->h.data || io->h_kept.q))
        return PTORED_ERR_INVALID_ARG;
    if (p.post_weight == nullptr && io->post_rstd) return PTORED_ERR_INVALID_ARG;
    if (p.pre_weight == nullptr && (io->z.data || io->z_kept.q || io->pre_rstd))
        return PTORED_ERR_INVALID_ARG;
    const int es = esize_of(p.dtype), ws = esize_of(p.weight_dtype);
    Buffers b;
    bool ok = b.rows(io->x.data, p.rows, p.cols, io->x.ld, es, false);
    for (int r = 0; r < nranks && ok; ++r)
        ok = parts[r] != nullptr && b.rows(parts[r], p.rows, p.cols, part_ld, es, false);
    ok = ok && b.rows(p.gate.data, p.gate_rows, p.cols, p.gate.ld, es, false, false) &&
         b.rows(io->x_out.data, p.rows, p.cols, io->x_out.ld, es, true) &&
         b.rows(io->z.data, p.rows, p.cols, io->z.ld, es, true) &&
         b.rows(io->h.data, p.rows, p.cols, io->h.ld, es, true) &&
         b.kept(io->h_kept, p.rows, p.cols, true) && b.kept(io->x_kept, p.rows, p.cols, true) &&
         b.kept(io->z_kept, p.rows, p.cols, true);
    if (!ok) return PTORED_ERR_INVALID_ARG;
    if (!params_supported(params)) return PTORED_ERR_UNSUPPORTED;
    b.vec(p.post_weight, p.cols * ws, ws, false);
    b.vec(p.pre_weight, p.cols * ws, ws, false);
    b.vec(io->post_rstd, p.rows * 4, 4, true);
    b.vec(io->pre_rstd, p.rows * 4, 4, true);
    if (!b.aligned()) return PTORED_ERR_INVALID_ARG;
    if (!b.disjoint()) return PTORED_ERR_OVERLAP;
    if (p.rows == 0 || p.cols == 0) return PTORED_OK;

    NormArgs a{};
    for (int r = 0; r < nranks; ++r) a.part[r] = static_cast<const char*>(parts[r]);
    a.part_ld = part_ld * es;
    a.nranks = nranks;
    a.rows = p.rows;
    a.cols = (int32_t)p.cols;
    a.x = mat(io->x, es);
    a.x_out = mat(io->x_out, es);
    a.z = mat(io->z, es);
    a.h = mat(io->h, es);
    a.gate = mat(p.gate, es);
    a.kh = kept(io->h_kept);
    a.kx = kept(io->x_kept);
    a.kz = kept(io->z_kept);
    a.w1 = static_cast<const char*>(p.post_weight);
    a.w2 = static_cast<const char*>(p.pre_weight);
    a.r1 = io->post_rstd;
    a.r2 = io->pre_rstd;
    a.rows_per_gate = p.gate.data ? p.rows / p.gate_rows : p.rows;
    a.w_f32 = p.weight_dtype == PTORED_F32;
    a.offset = p.weight_offset;
    a.alpha = p.branch_scale;
    a.beta = p.residual_scale;
    a.eps = p.eps;
    a.inv_cols = 1.0f / (float)p.cols;
    return status_of(PTORED_BY_TYPE(norm, p.dtype, a, stream));
}

extern "C" int ptored_block_norm_backward_workspace(int64_t rows, int64_t cols, int64_t gate_rows,
                                                    int64_t* bytes) {
    if (bytes == nullptr || !shape_ok(rows, cols) || gate_rows < 0 ||
        (gate_rows > 0 && rows % gate_rows != 0))
        return PTORED_ERR_INVALID_ARG;
    if (cols > PTORED_BLOCK_MAX_COLS) return PTORED_ERR_UNSUPPORTED;
    // of any type
    *bytes = std::max(grad_workspace(cols, gate_rows, grad_split(rows, cols, gate_rows, PTORED_F32)),
                      grad_workspace(cols, gate_rows, grad_split(rows, cols, gate_rows, PTORED_BF16)));
    return PTORED_OK;
}

extern "C" int ptored_block_norm_backward(const ptored_block_params* params,
                                          const ptored_block_grad_io* io, hipStream_t stream) {
    if (!params_valid(params) || io == nullptr) return PTORED_ERR_INVALID_ARG;
    const ptored_block_params& p = *params;
    const bool pre = p.pre_weight != nullptr, post = p.post_weight != nullptr;
    const bool need_h = post || io->dgate.data != nullptr;
    const int64_t gate_rows = p.gate.data ? p.gate_rows : 0;  // not read without a gate
    const bool packed = io->x_kept.q != nullptr || io->h_kept.q != nullptr;
    if (packed && (io->x_out.data || io->h.data)) return PTORED_ERR_INVALID_ARG;
    if (pre != (io->dz.data != nullptr) || (!pre && io->dx_out.data == nullptr))
        return PTORED_ERR_INVALID_ARG;
    if (pre && (io->pre_rstd == nullptr || !(packed ? io->x_kept.q : io->x_out.data)))
        return PTORED_ERR_INVALID_ARG;
    if (post && io->post_rstd == nullptr) return PTORED_ERR_INVALID_ARG;
    if (need_h && !(packed ? io->h_kept.q : io->h.data)) return PTORED_ERR_INVALID_ARG;
    if ((!post && io->dpost_weight) || (!pre && io->dpre_weight) ||
        (p.gate.data == nullptr && io->dgate.data))
        return PTORED_ERR_INVALID_ARG;
    const int es = esize_of(p.dtype), ws = esize_of(p.weight_dtype);
    Buffers b;
    const bool ok = b.rows(io->dz.data, p.rows, p.cols, io->dz.ld, es, false) &&
                    b.rows(io->dx_out.data, p.rows, p.cols, io->dx_out.ld, es, false) &&
                    b.rows(io->x_out.data, p.rows, p.cols, io->x_out.ld, es, false) &&
                    b.rows(io->h.data, p.rows, p.cols, io->h.ld, es, false) &&
                    b.rows(p.gate.data, gate_rows, p.cols, p.gate.ld, es, false, false) &&
                    b.kept(io->x_kept, p.rows, p.cols, false) &&
                    b.kept(io->h_kept, p.rows, p.cols, false) &&
                    b.rows(io->dx.data, p.rows, p.cols, io->dx.ld, es, true) &&
                    b.rows(io->dh.data, p.rows, p.cols, io->dh.ld, es, true) &&
                    b.rows(io->dgate.data, gate_rows, p.cols, io->dgate.ld, es, true, false);
    if (!ok) return PTORED_ERR_INVALID_ARG;
    if (!params_supported(params)) return PTORED_ERR_UNSUPPORTED;
    b.vec(p.post_weight, p.cols * ws, ws, false);
    b.vec(p.pre_weight, p.cols * ws, ws, false);
    b.vec(io->post_rstd, p.rows * 4, 4, false);
    b.vec(io->pre_rstd, p.rows * 4, 4, false);
    b.vec(io->dpost_weight, p.cols * ws, ws, true);
    b.vec(io->dpre_weight, p.cols * ws, ws, true);

    const bool gated = io->dgate.data != nullptr;
    // gate rows without a gradient: a chunk that walks several takes them in order
    const bool in_order = !gated && gate_rows > 1 && gate_rows < p.rows;
    const GradSplit split = grad_split(p.rows, p.cols, gated ? gate_rows : 0, p.dtype, in_order);
    GradArgs a{};
    // with its gradient wanted, a chunk lies within a gate row or begins with one
    const int64_t rows_per_gate = gate_rows > 0 ? p.rows / gate_rows : p.rows;
    const bool one = gated ? !split.gate_direct : gate_rows <= 1;
    a.chunk_gates = one ? kOneGate : rows_per_gate == 1 ? kEachGate : kSomeGates;
    a.gate_direct = split.gate_direct;
    a.gate_joined = gated && !split.gate_direct;
    a.gate_units = gate_rows > 1 ? 1 : 0;
    a.slot_w1 = a.slot_w2 = -1;
    if (io->dpost_weight || a.gate_joined) a.slot_w1 = a.ws_slots++;
    if (io->dpre_weight) a.slot_w2 = a.ws_slots++;
    a.ws_pitch = grad_pitch(p.cols);
    // as much as the query gives, which counts a row for each sum that is wanted
    const int wanted = (io->dpost_weight != nullptr) + (io->dpre_weight != nullptr) + a.gate_joined;
    const int64_t need = split.chunks * a.ws_pitch * 4 * wanted;
    if (need > 0 && (io->workspace == nullptr || io->workspace_bytes < need))
        return PTORED_ERR_INVALID_ARG;
    if (need > 0) b.vec(io->workspace, need, 16, true);
    if (!b.aligned()) return PTORED_ERR_INVALID_ARG;
    if (!b.disjoint()) return PTORED_ERR_OVERLAP;
    if (p.cols == 0) return PTORED_OK;

    a.rows = p.rows;
    a.cols = (int32_t)p.cols;
    a.dz = mat(io->dz, es);
    a.dxo = mat(io->dx_out, es);
    a.x = mat(io->x_out, es);
    a.h = mat(io->h, es);
    a.dx = mat(io->dx, es);
    a.dh = mat(io->dh, es);
    a.gate = mat(p.gate, es);
    a.dgate = mat(io->dgate, es);
    a.kx = kept(io->x_kept);
    a.kh = kept(io->h_kept);
    a.w1 = static_cast<const char*>(p.post_weight);
    a.w2 = static_cast<const char*>(p.pre_weight);
    a.r1 = io->post_rstd;
    a.r2 = io->pre_rstd;
    a.ws = static_cast<float*>(io->workspace);
    a.dw1 = static_cast<char*>(io->dpost_weight);
    a.dw2 = static_cast<char*>(io->dpre_weight);
    a.unit_rows = split.unit_rows;
    a.chunks_per_unit = split.chunks_per_unit;
    a.chunk_rows = split.chunk_rows;
    a.chunk_first = split.chunk_first;
    a.row_step = split.row_step;
    a.chunks = split.chunks;
    a.gate_rows = gate_rows;
    a.rows_per_gate = rows_per_gate;
    a.w_f32 = p.weight_dtype == PTORED_F32;
    a.offset = p.weight_offset;
    a.alpha = p.branch_scale;
    a.beta = p.residual_scale;
    a.inv_cols = 1.0f / (float)p.cols;
    return status_of(PTORED_BY_TYPE(grad, p.dtype, a, stream));
}

extern "C" int ptored_checkpoint_pack(ptored_rows x, int64_t rows, int64_t cols, int dtype,
                                      ptored_checkpoint k, hipStream_t stream) {
    const int st = checkpoint_args(x, rows, cols, dtype, k, true);
    if (st != PTORED_OK || rows == 0 || cols == 0) return st;
    const PackArgs a{mat(x, esize_of(dtype)), kept(k), rows, (int32_t)cols};
    return status_of(PTORED_BY_TYPE(pack, dtype, a, stream));
}

extern "C" int ptored_checkpoint_unpack(ptored_checkpoint k, int64_t rows, int64_t cols, int dtype,
                                        ptored_rows out, hipStream_t stream) {
    const int st = checkpoint_args(out, rows, cols, dtype, k, false);
    if (st != PTORED_OK || rows == 0 || cols == 0) return st;
    const PackArgs a{mat(out, esize_of(dtype)), kept(k), rows, (int32_t)cols};
    return status_of(PTORED_BY_TYPE(unpack, dtype, a, stream));
}

extern "C" int ptored_checkpoint_wgrad_workspace(int64_t rows, int64_t outs, int64_t cols,
                                                 int dtype, int64_t* bytes) {
    if (bytes == nullptr || !shape_ok(rows, outs) || !shape_ok(rows, cols) ||
        !shape_ok(outs, cols))
        return PTORED_ERR_INVALID_ARG;
    if (!float_type(dtype)) return PTORED_ERR_UNSUPPORTED;
    *bytes = wgrad_workspace(outs, cols, wgrad_shape(rows, outs, cols, dtype));
    return PTORED_OK;
}

extern "C" int ptored_checkpoint_wgrad(ptored_rows dy, ptored_checkpoint x, int64_t rows,
                                       int64_t outs, int64_t cols, int dtype, ptored_rows dw,
                                       int dw_dtype, int accumulate, void* workspace,
                                       int64_t workspace_bytes, hipStream_t stream) {
    if (dy.data == nullptr || x.q == nullptr || dw.data == nullptr) return PTORED_ERR_INVALID_ARG;
    if (!shape_ok(rows, outs) || !shape_ok(rows, cols) || !shape_ok(outs, cols) ||
        outs > kMaxCols || cols > kMaxCols)
        return PTORED_ERR_INVALID_ARG;
    Buffers b;
    if (!b.rows(dy.data, rows, outs, dy.ld, esize_of(dtype), false) ||
        !b.kept(x, rows, cols, false) ||
        !b.rows(dw.data, outs, cols, dw.ld, esize_of(dw_dtype), true))
        return PTORED_ERR_INVALID_ARG;
    if (!float_type(dtype) || (dw_dtype != PTORED_F32 && dw_dtype != dtype))
        return PTORED_ERR_UNSUPPORTED;
    const WgradShape w = wgrad_shape(rows, outs, cols, dtype);
    // a launch takes fewer than 2^32 threads
    if (w.tiles_m * w.tiles_n > int64_t(1) << 22) return PTORED_ERR_UNSUPPORTED;
    const int64_t need = wgrad_workspace(outs, cols, w);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return PTORED_ERR_INVALID_ARG;
    if (need > 0) b.vec(workspace, need, 16, true);
    if (!b.aligned()) return PTORED_ERR_INVALID_ARG;
    // dw is read only as itself: no exact alias with dy
    if (!b.disjoint() || dy.data == dw.data) return PTORED_ERR_OVERLAP;
    if (outs == 0 || cols == 0 || (rows == 0 && accumulate)) return PTORED_OK;

    WgradArgs a{};
    a.dy = static_cast<const char*>(dy.data);
    a.dy_ld = dy.ld * esize_of(dtype);
    a.x = kept(x);
    a.dw = static_cast<char*>(dw.data);
    a.dw_ld = dw.ld * esize_of(dw_dtype);
    a.ws = static_cast<float*>(workspace);
    a.rows = rows;
    a.rows_per_split = w.rows_per_split;
    a.outs = (int32_t)outs;
    a.cols = (int32_t)cols;
    a.splits = (int32_t)w.splits;
    a.dw_f32 = dw_dtype == PTORED_F32;
    a.accumulate = accumulate != 0;
    a.tiles_m = (int32_t)w.tiles_m;
    a.tiles_n = (int32_t)w.tiles_n;
    a.shape = w.shape;
    a.ws_ld = wgrad_pitch(cols);
    return status_of(PTORED_BY_TYPE(wgrad, dtype, a, stream));
}
