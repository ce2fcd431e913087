// extents.cpp -- what the C ABI's host code takes for an overlap of two buffers, byte
// by byte: built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_extents_cpu.py with tests/sanitize/step_stub.cpp instead of the
// kernels; needs no GPU.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "block/block_checks.hpp"
#include "step_stub.h"

using namespace ptored::step;
using ptored::block::Extent;
using ptored::block::extent_of;

namespace {

#define EXPECT(what, ...)                                                  \
    do {                                                                   \
        if (!(what)) {                                                     \
            std::printf("FAIL %s: ", #what), std::printf(__VA_ARGS__);     \
            std::printf("\n");                                             \
            return 1;                                                      \
        }                                                                  \
    } while (0)

struct Matrix {
    int64_t at, rows, cols, ld;
    int es;
};

// The bytes that a matrix holds, in a small memory.
std::vector<bool> bytes_of(const Matrix& m) {
    std::vector<bool> on(2000);
    for (int64_t r = 0; r < m.rows; ++r)
        for (int64_t b = 0; b < m.cols * m.es; ++b) on[(size_t)(m.at + r * m.ld * m.es + b)] = true;
    return on;
}

int pairs() {
    std::mt19937_64 rng(3);
    int between = 0, shared = 0, counted = 0;
    for (int i = 0; i < 100000; ++i) {
        Matrix m[2];
        for (Matrix& v : m) {
            v.es = rng() % 2 ? 2 : 4;
            v.rows = (int64_t)(rng() % 7);
            v.cols = (int64_t)(rng() % 9);
            v.ld = v.cols + (rng() % 3 ? (int64_t)(rng() % 14) : 0);
            v.at = 256 + (int64_t)(rng() % 120);
        }
        if (rng() % 2) {
            m[1].es = m[0].es;
            m[1].ld = std::max(m[1].cols, m[0].ld);
        }
        Extent e[2];
        for (int k = 0; k < 2; ++k)
            e[k] = extent_of(reinterpret_cast<void*>(0x10000 + m[k].at), m[k].rows, m[k].cols,
                             m[k].rows > 1 ? m[k].ld : m[k].cols, m[k].es);
        const std::vector<bool> a = bytes_of(m[0]), b = bytes_of(m[1]);
        bool want = false;
        for (size_t k = 0; k < a.size(); ++k) want = want || (a[k] && b[k]);
        const bool got = meet(e[0], e[1]);
        EXPECT(got == meet(e[1], e[0]), "either way round");
        EXPECT(got || !want, "pair %d shares a byte", i);
        if (got && !want) {
            // both in rows with gaps, of different pitches
            EXPECT(e[0].width < e[0].bytes && e[1].width < e[1].bytes && e[0].pitch != e[1].pitch, "pair %d", i);
            ++counted;
        }
        between += !got && spans_meet(e[0], e[1]);
        shared += want;
    }
    EXPECT(between > 3000 && shared > 25000 && counted > 300, "%d %d %d", between, shared, counted);
    // addresses and pitches near the largest
    const int64_t far = int64_t(1) << 58;
    const Extent x = extent_of(reinterpret_cast<void*>(64), 4, 8, far, 4), y = extent_of(reinterpret_cast<void*>(96), 4, 8, far, 4);
    EXPECT(spans_meet(x, y) && !meet(x, y) && !meet(y, x), "far rows");
    EXPECT(meet(x, extent_of(reinterpret_cast<void*>(92), 4, 8, far, 4)), "far rows that meet");
    return 0;
}

// Calls on halves of a buffer are made; a column more, and they are refused.
int halves() {
    auto at = [](int k, int64_t elem = 0) { return reinterpret_cast<char*>((uintptr_t)(k + 1) << 36) + elem * 2; };
    const int64_t T = 300, D = 264, F = 136;
    for (const int64_t more : {0, 1}) {
        const int want = more ? PTORED_ERR_OVERLAP : PTORED_OK;
        const ptored_ffn_params p{T, D, F, PTORED_BF16, 0};
        const ptored_rows x{at(1), D}, wg{at(2), D}, wu{at(3), D}, y{at(4), F};
        const ptored_rows gate{at(5), 2 * F}, up{at(5, F - more), 2 * F};
        void* const ws = at(20);
        g_seen = {};
        EXPECT(ptored_gated_ffn(&p, x, wg, wu, y, gate, up, ws, 1 << 30, nullptr) == want, "forward");
        EXPECT(g_seen.products.size() == (size_t)(1 - more), "forward's launch");
        ptored_ffn_grad_io io{};
        io.dy = y;
        io.gate = io.dgate = gate;
        io.up = io.dup = up;
        io.x = {at(6), 2 * D};
        io.dx = {at(6, D - more), 2 * D};
        io.w_gate = wg;
        io.w_up = wu;
        io.dw_gate = {at(7), 2 * D};
        io.dw_up = {at(7, D - more), 2 * D};
        io.dw_dtype = PTORED_BF16;
        io.workspace = ws;
        io.workspace_bytes = 1 << 30;
        EXPECT(ptored_gated_ffn_backward(&p, &io, nullptr) == want, "backward");
        const ptored_layer_norm_params n{T, D, nullptr, nullptr, 0, PTORED_BF16, PTORED_F32};
        EXPECT(ptored_layer_norm(nullptr, 0, D, &n, x, {at(8), 2 * D}, {at(8, D - more), 2 * D}, nullptr, nullptr,
                                 nullptr) == want, "layer norm");
        // statistics behind a single row, and between rows
        float* const stat = reinterpret_cast<float*>(at(9, D + 2 - 4 * more));
        const ptored_layer_norm_params one{1, D, nullptr, nullptr, 0, PTORED_BF16, PTORED_F32};
        EXPECT(ptored_layer_norm(nullptr, 0, D, &one, x, {}, {at(9), D}, stat, nullptr, nullptr) == want, "behind");
        const ptored_layer_norm_params two{2, D, nullptr, nullptr, 0, PTORED_BF16, PTORED_F32};
        EXPECT(ptored_layer_norm(nullptr, 0, D, &two, x, {}, {at(9), 2 * D}, stat, nullptr, nullptr) == want, "between");
    }
    return 0;
}

// Column slices of one gradient, each scaled in place or into slices of another; one
// a column too wide, and the call is refused.
int slices() {
    std::mt19937_64 rng(4);
    for (int i = 0; i < 4000; ++i) {
        const int count = 1 + (int)(rng() % (i % 10 ? 6 : 200));
        const int64_t rows = 2 + (int64_t)(rng() % 5);
        std::vector<int64_t> width((size_t)count), first((size_t)count);
        int64_t cols = 0;
        for (size_t k = 0; k < width.size(); ++k) {
            cols += (int64_t)(rng() % 3);
            first[k] = cols;
            cols += width[k] = 1 + (int64_t)(rng() % 40);
        }
        const int64_t ld = cols + (int64_t)(rng() % 3);
        const bool into = rng() % 2;
        const int dtype = (int)(rng() % 3), es = dtype == PTORED_F32 ? 4 : 2;
        const int out_dtype = into && rng() % 2 ? PTORED_F32 : dtype, oes = out_dtype == PTORED_F32 ? 4 : 2;
        char *data = reinterpret_cast<char*>((uintptr_t)1 << 40), *out = reinterpret_cast<char*>((uintptr_t)2 << 40);
        std::vector<ptored_grad> g((size_t)count + 1);
        for (size_t k = 0; k < width.size(); ++k)
            g[k] = {data + first[k] * es, into ? out + first[k] * oes : data + first[k] * es, rows, width[k], ld, ld,
                    dtype, out_dtype};
        g.back() = {nullptr, nullptr, 0, INT64_MAX / 2, INT64_MAX, INT64_MAX, dtype, dtype};  // of no rows: not read
        std::shuffle(g.begin(), g.end(), rng);
        int64_t need = 0;
        EXPECT(ptored_grad_norm_workspace(g.data(), count + 1, &need) == PTORED_OK, "query");
        void* const ws = reinterpret_cast<void*>((uintptr_t)3 << 40);
        float* const norm = reinterpret_cast<float*>((uintptr_t)4 << 40);
        EXPECT(ptored_grad_clip(g.data(), count + 1, 1.0f, norm, ws, need, nullptr) == PTORED_OK, "%d slices", count);
        EXPECT(ptored_grad_norm(g.data(), count + 1, norm, ws, need, nullptr) == PTORED_OK, "%d slices", count);
        // one reaches into the next, its last column behind the buffer's into the next row's first
        size_t k = rng() % g.size();
        if (g[k].rows == 0) k = (k + 1) % g.size();
        int64_t to = ld;
        for (const ptored_grad& e : g)
            if (e.rows > 0 && e.data > g[k].data)
                to = std::min(to, ((const char*)e.data - (const char*)g[k].data) / es);
        const int64_t at = ((const char*)g[k].data - data) / es;
        if (to == ld && (count == 1 || ld - at + first[0] >= ld)) continue;
        g[k].cols = to == ld ? ld - at + first[0] + 1 : to + 1;
        if (g[k].cols > ld) continue;
        EXPECT(ptored_grad_clip(g.data(), count + 1, 1.0f, norm, ws, need + 4096, nullptr) == PTORED_ERR_OVERLAP,
               "%d slices, one too wide", count);
    }
    // the norm beside a single column, and on it
    float* const m = reinterpret_cast<float*>((uintptr_t)1 << 40);
    const ptored_grad column{m, m, 9, 1, 4, 4, PTORED_F32, PTORED_F32};
    void* const ws = reinterpret_cast<void*>((uintptr_t)3 << 40);
    for (int k = 0; k < 8; ++k) {
        const int want = k % 4 ? PTORED_OK : PTORED_ERR_OVERLAP;
        EXPECT(ptored_grad_clip(&column, 1, 1.0f, m + k, ws, 64, nullptr) == want, "norm at %d", k);
        EXPECT(ptored_grad_norm(&column, 1, m + k, ws, 64, nullptr) == want, "norm at %d", k);
    }
    return 0;
}

}  // namespace

int main() { return pairs() || halves() || slices() ? 1 : (std::printf("ok\n"), 0); }
