// step_launches.cpp -- drives the host code of the step's operators through the C
// ABI with made-up device addresses, linked against tests/sanitize/step_stub.cpp
// instead of the kernels.  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_step_launches_cpu.py, which runs one
// check at a time (by name); needs no GPU.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "step_stub.h"

using namespace ptored::step;

namespace {

#define EXPECT(what, ...)                                     \
    do {                                                      \
        if (!(what)) {                                        \
            std::printf("FAIL %s: ", #what), std::printf(__VA_ARGS__); \
            std::printf("\n");                                \
            return 1;                                         \
        }                                                     \
    } while (0)

// Fake device address of buffer k, 64 GiB apart.
void* fake(int k) { return reinterpret_cast<void*>((uintptr_t)(k + 1) << 36); }
ptored_rows mat(int k, int64_t ld) { return {fake(k), ld}; }

struct Tile {
    int64_t rows, cols;
    bool f32, narrow, held, direct;  // types and ways in which there is one
};
Tile tile_of(int shape) {
    switch (shape) {
        case kTile128: return {128, 128, true, true, true, true};
        case kTile128Deep: return {128, 128, true, true, false, true};
        case kTile256: return {256, 256, false, true, true, true};
        case kTile64: return {64, 64, false, true, false, true};
        case kTile128x32: return {128, 64, true, true, false, true};
        case kTile32x128: return {32, 128, true, true, true, true};
        case kTile64x128: return {64, 128, true, true, true, true};
        case kTileShort: return {128, 128, true, true, true, false};
        default: return {256, 128, true, false, true, true};  // kTileSplit
    }
}

// One launch: its tiles cover the output, its splits every step, its partial sums
// lie in the workspace.
int look(const Product& p, int64_t workspace) {
    const ProductArgs& a = p.a;
    const int es = p.dtype == PTORED_F32 ? 4 : 2;
    const int64_t outs = p.kind == kForward ? 2 : a.outs;
    EXPECT(a.splits >= 1, "splits");
    if (a.splits > 1)
        EXPECT(a.ws_ld % 4 == 0 && a.ws_ld >= a.n &&
                   reinterpret_cast<char*>(a.ws) + a.splits * outs * a.m * a.ws_ld * 4 <=
                       static_cast<char*>(fake(12)) + workspace,
               "%d splits of %lld x %lld", a.splits, (long long)a.m, (long long)a.n);
    if (a.shape >= kFew16) {
        const int64_t tokens = a.shape == kFew16 ? 16 : a.shape == kFew32 ? 32 : 64;
        const int64_t features = a.shape == kFew64 ? 32 : 16;
        EXPECT(p.kind == kForward && a.m <= tokens && a.k * es >= 16, "few");
        EXPECT(a.shape == kFew16 || p.dtype == PTORED_F32, "few's type");
        EXPECT(a.tiles_n * features >= a.n && (a.tiles_n - 1) * features < a.n, "few's tiles");
        EXPECT(a.waves == 8 || (a.waves == 16 && a.shape == kFew16), "few's waves");
        return 0;
    }
    const Tile t = tile_of(a.shape);
    EXPECT(p.dtype == PTORED_F32 ? t.f32 : t.narrow, "shape %d of type %d", a.shape, p.dtype);
    EXPECT(a.direct ? t.direct : t.held, "shape %d, direct %d", a.shape, a.direct);
    const int64_t least = p.kind == kForward ? a.k : std::min(a.n, p.kind == kInput ? a.k : a.m);
    EXPECT((least * es < 16) == (a.shape == kTileShort), "rows of %lld elements", (long long)least);
    EXPECT(p.kind == kInput || a.shape != kTile32x128, "kind");
    EXPECT(p.kind == kForward || (a.shape != kTile64 && a.shape != kTile128x32), "kind");
    EXPECT(p.kind != kWeight || a.shape != kTile64x128, "kind");
    const int64_t cols = p.kind == kForward ? t.cols / 2 : t.cols;
    EXPECT(a.tiles_m * t.rows >= a.m && (a.tiles_m - 1) * t.rows < a.m, "rows");
    EXPECT(a.tiles_n * cols >= a.n && (a.tiles_n - 1) * cols < a.n, "columns");
    const int64_t depth = kStepBytes / es;
    const int64_t steps = std::max<int64_t>(1, (a.k + depth - 1) / depth) * (p.kind == kInput ? 2 : 1);
    EXPECT(a.steps_per_split * a.splits >= steps && a.steps_per_split * (a.splits - 1) < steps,
           "%d splits of %lld of %lld steps", a.splits, (long long)a.steps_per_split, (long long)steps);
    EXPECT((int64_t)a.tiles_m * a.tiles_n * a.outs * a.splits <= int64_t(1) << 22, "launch");
    // operands' pitches, and those of single rows
    for (int i = 0; i < 2; ++i)
        EXPECT(a.a_ld[i] >= 0 && a.a_ld[i] <= PTORED_FFN_MAX_PITCH && a.b_ld[i] >= 0 &&
                   a.b_ld[i] <= PTORED_FFN_MAX_PITCH, "pitches");
    if (a.direct)
        for (int i = 0; i < 2; ++i)
            EXPECT(a.a_ld[i] % 16 == 0 && a.b_ld[i] % 16 == 0, "direct pitches");
    return 0;
}

int products() {
    std::mt19937_64 rng(1);
    auto size = [&](int64_t most) {
        const double u = std::uniform_real_distribution<double>(0, 1)(rng);
        int64_t n = (int64_t)(std::pow((double)most, u) + 0.5);
        const int kind = (int)(rng() % 3);
        if (kind == 0) n = n / 64 * 64;
        if (kind == 1) n = n / 8 * 8;
        return std::max<int64_t>(1, n);
    };
    int both = 0;
    for (int i = 0; i < 20000; ++i) {
        const int dtype = (int)(rng() % 3);
        const int64_t T = size(70000), D = size(20000), F = size(20000), pad = (int64_t)(rng() % 3) * 4;
        const ptored_ffn_params p{T, D, F, dtype, 0};
        int64_t need = 0;
        EXPECT(ptored_gated_ffn_workspace(T, D, F, dtype, &need) == PTORED_OK, "query");
        g_seen = {};
        // a single row's pitch is any
        const int64_t x_ld = T == 1 ? (int64_t)1 << 50 : D + pad;
        int st = ptored_gated_ffn(&p, mat(1, x_ld), mat(2, D + pad), mat(3, D + pad), mat(4, F), mat(5, F),
                                  mat(6, F), fake(12), need, nullptr);
        EXPECT(st == PTORED_OK && g_seen.products.size() == 1, "%lld %lld %lld: %d", (long long)T,
               (long long)D, (long long)F, st);
        if (look(g_seen.products[0], need)) return 1;
        EXPECT(ptored_gated_ffn_backward_workspace(T, D, F, dtype, &need) == PTORED_OK, "query");
        ptored_ffn_grad_io io{};
        io.dy = mat(1, F);
        io.gate = mat(2, F);
        io.up = mat(3, F);
        io.dgate = mat(4, T == 1 ? (int64_t)1 << 50 : F + pad);
        io.dup = mat(5, F);
        io.x = mat(6, x_ld);
        io.w_gate = mat(7, D);
        io.w_up = mat(8, D + pad);
        const int which = 1 + (int)(rng() % 7);
        if (which & 1) io.dx = mat(9, D);
        if (which & 2) io.dw_gate = mat(10, D);
        if (which & 4) io.dw_up = mat(11, D);
        io.dw_dtype = dtype;
        io.workspace = fake(12);
        io.workspace_bytes = need;
        g_seen = {};
        st = ptored_gated_ffn_backward(&p, &io, nullptr);
        EXPECT(st == PTORED_OK, "%lld %lld %lld: %d", (long long)T, (long long)D, (long long)F, st);
        EXPECT(g_seen.products.size() == (size_t)((which & 1) + (which > 1)) && g_seen.others == 1, "launches");
        for (const Product& q : g_seen.products)
            if (look(q, need)) return 1;
        if (g_seen.firsts.empty()) continue;
        ++both;
        const ProductArgs &w = g_seen.products[0].a, &d = g_seen.products[1].a;
        EXPECT(g_seen.products.size() == 2 && w.shape == kTile128 && d.shape == kTile128 && w.direct == d.direct,
               "both");
        EXPECT(g_seen.firsts[0] == w.tiles_m * w.tiles_n * w.outs * w.splits, "the weights' workgroups");
        if (w.splits > 1 && d.splits > 1)
            EXPECT(d.ws >= w.ws + w.splits * w.outs * w.m * w.ws_ld, "partial sums of both");
    }
    EXPECT(both > 1000, "%d launches of both gradients", both);
    return 0;
}

int layers() {
    for (int64_t rows : {1, 2, 255, 256, 300, 5000, 100000, 900000})
        for (int64_t cols : {1, 7, 64, 1000, 4096, 8200, 16384})
            for (int dtype = 0; dtype < 3; ++dtype) {
                int64_t need = 0;
                EXPECT(ptored_layer_norm_backward_workspace(rows, cols, &need) == PTORED_OK, "query");
                ptored_layer_norm_params p{rows, cols, nullptr, nullptr, 0, dtype, PTORED_F32};
                g_seen = {};
                const int st = ptored_layer_norm_backward(
                    &p, mat(1, cols), mat(2, cols), mat(3, cols), static_cast<float*>(fake(4)),
                    static_cast<float*>(fake(5)), mat(6, cols), fake(7), fake(8), fake(9), need, nullptr);
                EXPECT(st == PTORED_OK && g_seen.layers.size() == 1, "%lld x %lld", (long long)rows,
                       (long long)cols);
                const LayerGradArgs& a = g_seen.layers[0];
                EXPECT(a.chunks >= 1 && a.chunks <= rows && a.chunks <= 5120, "chunks");
                EXPECT(a.ws_pitch % 4 == 0 && a.ws_pitch >= cols && a.chunks * 2 * a.ws_pitch * 4 <= need,
                       "workspace");
            }
    return 0;
}

// The entries that a pack stands for, as the kernel reads it.
std::vector<GradEntry> unpack(const GradPack& p) {
    std::vector<GradEntry> out;
    for (int i = 0; i < p.slots; ++i) {
        if (!(p.heads[i / 32] >> (i % 32) & 1)) continue;
        GradEntry e{};
        const uint64_t d = p.data[i];
        e.data = reinterpret_cast<const char*>(d & 0xFFFFFFFFFFFFull);
        e.out = reinterpret_cast<char*>(p.out[i]);
        e.cols = (int64_t)((d >> 48 & 0xFF) << 32 | p.cols[i]);
        e.rows = 1;
        const int type = (int)(d >> 56 & 7);
        e.type = type > PTORED_F16 ? type - 3 : type | type << 8;
        if (d >> 59 & 1) {
            e.rows = (int32_t)(uint32_t)p.data[i + 1];
            e.ld = (int32_t)(p.data[i + 1] >> 32);
            e.out_ld = (int32_t)p.out[i + 1];
        }
        out.push_back(e);
    }
    return out;
}

int gradients() {
    std::mt19937_64 rng(2);
    for (int i = 0; i < 3000; ++i) {
        const int count = (int)(rng() % 5 == 0 ? rng() % 900 : rng() % 90);
        std::vector<ptored_grad> g((size_t)count);
        for (int k = 0; k < count; ++k) {
            ptored_grad& e = g[(size_t)k];
            e.data = reinterpret_cast<void*>(((uintptr_t)1 << 40) + ((uintptr_t)k << 34));
            e.out = rng() % 2 ? const_cast<void*>(e.data)
                              : reinterpret_cast<void*>(((uintptr_t)1 << 45) + ((uintptr_t)k << 34));
            e.rows = rng() % 3 == 0 ? (int64_t)(rng() % 300) : 1;
            e.cols = (int64_t)(rng() % 7 == 0 ? rng() % 3 : rng() % 20000);
            e.ld = e.out_ld = e.cols + (int64_t)(rng() % 9);
            e.dtype = (int)(rng() % 3);
            e.out_dtype = e.out != e.data && rng() % 2 ? PTORED_F32 : e.dtype;
        }
        int64_t need = 0;
        EXPECT(ptored_grad_norm_workspace(g.data(), count, &need) == PTORED_OK, "query");
        char* const ws = static_cast<char*>(fake(9000));
        float* const norm = static_cast<float*>(fake(9001));
        g_seen = {};
        const int st = ptored_grad_clip(g.data(), count, 1.0f, norm, ws, need, nullptr);
        EXPECT(st == PTORED_OK, "%d gradients: %d", count, st);
        std::vector<const ptored_grad*> want;
        for (const ptored_grad& e : g)
            if (e.rows > 0 && e.cols > 0) want.push_back(&e);
        if (want.empty()) {
            EXPECT(g_seen.joins.size() == 1 && g_seen.joins[0].all_count == 0 && g_seen.sums.empty() &&
                       g_seen.scales.empty(), "nothing to do");
            continue;
        }
        EXPECT(g_seen.sums.size() == 1 && g_seen.scales.size() == 1 && g_seen.joins.empty(), "launches");
        const GradList& s = g_seen.sums[0];
        const GradList& t = g_seen.scales[0];
        std::vector<GradEntry> got;
        int64_t table = 0;
        if (want.size() > (size_t)kGradEntries) {
            int64_t chunks = 0;
            for (const GradPack& p : g_seen.packs) {
                EXPECT(p.first == chunks && reinterpret_cast<char*>(p.table) == ws + table, "a pack's place");
                for (GradEntry e : unpack(p)) {
                    e.first = (int32_t)chunks;
                    chunks += grad_chunks(e.rows, e.cols, e.type & 0xFF);
                    got.push_back(e);
                    table += (int64_t)sizeof(GradEntry);
                }
            }
            EXPECT(reinterpret_cast<const char*>(s.table) == ws && s.table == t.table, "table");
        } else {
            EXPECT(g_seen.packs.empty() && s.table == nullptr, "no table");
            got.assign(s.e, s.e + s.count);
        }
        EXPECT(got.size() == want.size() && s.count == (int)want.size(), "entries");
        int64_t chunks = 0;
        for (size_t k = 0; k < got.size(); ++k) {
            const GradEntry& e = got[k];
            const ptored_grad& w = *want[k];
            EXPECT(e.data == w.data && e.out == w.out && e.rows == w.rows && e.cols == w.cols &&
                       e.type == (w.dtype | w.out_dtype << 8) && e.first == chunks, "entry %zu", k);
            EXPECT(w.rows == 1 || (e.ld == w.ld && e.out_ld == w.out_ld), "pitches of %zu", k);
            chunks += grad_chunks(w.rows, w.cols, w.dtype);
        }
        EXPECT(s.chunks == chunks && t.chunks == chunks, "chunks");
        EXPECT(s.groups == std::min<int64_t>(chunks, kGradGroups) && t.groups == s.groups, "groups");
        EXPECT(reinterpret_cast<char*>(s.sums) == ws + table && t.all == s.sums && t.all_count == s.groups &&
                   table + s.groups * 8 <= need, "partial sums");
    }
    return 0;
}

}  // namespace

int main(int argc, char** argv) {
    const struct {
        const char* name;
        int (*check)();
    } checks[] = {{"products", products}, {"layers", layers}, {"gradients", gradients}};
    for (const auto& c : checks)
        if (argc == 2 && std::strcmp(argv[1], c.name) == 0) return c.check();
    std::printf("no such check\n");
    return 2;
}
