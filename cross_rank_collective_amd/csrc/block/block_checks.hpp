// block_checks.hpp -- argument checks that the C ABI's host code shares: shapes,
// pitches, alignment and overlaps of a call's buffers.
#pragma once

#include <cstdint>

#include "block_plan.h"

namespace ptored {
namespace block {

constexpr int64_t kMaxElems = int64_t(1) << 60;
constexpr int64_t kMaxCols = int64_t(1) << 30;

inline int esize_of(int dtype) { return dtype == PTORED_F32 ? 4 : 2; }
inline bool float_type(int dtype) { return dtype >= PTORED_F32 && dtype <= PTORED_F16; }

inline bool shape_ok(int64_t rows, int64_t cols) {
    return rows >= 0 && cols >= 0 && (cols == 0 || rows <= kMaxElems / cols);
}
// A pitch that holds the columns and whose byte extent fits.
inline bool pitch_ok(int64_t rows, int64_t cols, int64_t ld) {
    return ld >= cols && (ld == 0 || rows <= kMaxElems / ld);
}
inline int64_t blocks_of(int64_t cols) {
    return (cols + PTORED_CHECKPOINT_BLOCK - 1) / PTORED_CHECKPOINT_BLOCK;
}

// Where a buffer lies: rows of `width` bytes, one every `pitch`, `bytes` from the
// first to the end of the last.  One run of bytes is a row as wide as all of them.
struct Extent {
    uintptr_t p;
    int64_t bytes, pitch, width;
};
inline Extent extent_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int es) {
    const int64_t bytes = rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * es : 0;
    return {reinterpret_cast<uintptr_t>(p), bytes, ld * es, rows > 1 && ld > cols ? cols * es : bytes};
}
inline bool spans_meet(const Extent& a, const Extent& b) {
    return a.bytes > 0 && b.bytes > 0 && a.p < b.p + (uintptr_t)b.bytes && b.p < a.p + (uintptr_t)a.bytes;
}
// Whether two buffers share a byte.  Rows of one pitch, or of one buffer and a run,
// may lie between each other's; of different pitches they count as shared.
inline bool meet(const Extent& a, const Extent& b) {
    if (!spans_meet(a, b)) return false;
    const bool run_a = a.width == a.bytes, run_b = b.width == b.bytes;
    if (run_a && run_b) return true;
    if (run_a || run_b) {
        const Extent &run = run_a ? a : b, &rows = run_a ? b : a;
        const int64_t from = (int64_t)(run.p - rows.p);
        // the first row that ends behind the run's beginning
        const int64_t row = from < rows.width ? 0 : (from - rows.width) / rows.pitch + 1;
        return row * rows.pitch < rows.bytes && row * rows.pitch < from + run.bytes;
    }
    if (a.pitch != b.pitch) return true;
    // where the later one's rows begin between the earlier one's: either's bytes before
    // the other's (the spans meet, so there is a row to run into)
    const Extent &lo = a.p <= b.p ? a : b, &hi = a.p <= b.p ? b : a;
    const int64_t at = (int64_t)((hi.p - lo.p) % (uintptr_t)lo.pitch);
    return at < lo.width || at + hi.width > lo.pitch;
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
        add(extent_of(p, n, cols, n > 1 ? ld : cols, es), es, out, whole);
        return true;
    }
    bool kept(const ptored_checkpoint& k, int64_t n, int64_t cols, bool out) {
        if (k.q == nullptr) return true;
        if (k.scales == nullptr) return false;
        const int64_t nb = blocks_of(cols);
        if (!pitch_ok(n, cols, k.q_ld) || !pitch_ok(n, nb, k.scales_ld)) return false;
        add(extent_of(k.q, n, cols, k.q_ld, 1), 1, out, false);
        add(extent_of(k.scales, n, nb, k.scales_ld, 1), 1, out, false);
        return true;
    }
    void vec(const void* p, int64_t bytes, int align, bool out) {
        if (p != nullptr) add({reinterpret_cast<uintptr_t>(p), bytes, 0, bytes}, align, out, false);
    }
    bool aligned() const {
        for (int i = 0; i < n_; ++i)
            if (b_[i].at.p % (uintptr_t)b_[i].align != 0) return false;
        return true;
    }
    // No output overlaps another buffer, but for one that is exactly an input
    // matrix (gates and their gradients apart): same address, pitch and element size.
    bool disjoint() const {
        for (int i = 0; i < n_; ++i) {
            if (!b_[i].out) continue;
            for (int j = 0; j < n_; ++j) {
                const Buf &o = b_[i], &x = b_[j];
                if (i == j || !meet(o.at, x.at)) continue;
                const bool same = !x.out && o.matrix && x.matrix && o.at.p == x.at.p &&
                                  o.at.pitch == x.at.pitch && o.align == x.align;
                if (!same) return false;
            }
        }
        return true;
    }

  private:
    struct Buf {
        Extent at;
        int align;
        bool out, matrix;
    };
    void add(const Extent& at, int align, bool out, bool matrix) { b_[n_++] = {at, align, out, matrix}; }
    Buf b_[PTORED_MAX_RANKS + 24];
    int n_ = 0;
};

inline Mat mat(const ptored_rows& r, int es) { return {static_cast<char*>(r.data), r.ld * es}; }
inline Kept kept(const ptored_checkpoint& k) {
    return {static_cast<int8_t*>(k.q), k.q_ld, static_cast<uint8_t*>(k.scales), k.scales_ld};
}

inline int status_of(int rc) { return rc == kOk ? PTORED_OK : PTORED_ERR_HIP; }

#define PTORED_BY_TYPE(f, dtype, ...)                            \
    ((dtype) == PTORED_F32    ? f##_f32(__VA_ARGS__)             \
     : (dtype) == PTORED_BF16 ? f##_bf16(__VA_ARGS__)            \
                              : f##_f16(__VA_ARGS__))

}  // namespace block
}  // namespace ptored
