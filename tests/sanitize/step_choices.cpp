// step_choices.cpp -- which kernels the host code of the feed-forward block takes,
// linked against tests/sanitize/step_stub.cpp instead of the kernels, for
// tests/test_step_choices_cpu.py; needs no GPU.
//
//     step_choices cases < lines    each line "dtype rows cols wide pad call": the
//                                   kernels of that call, on a line of their own
//     step_choices all N            those of N drawn calls, each kernel once, with
//                                   the case of the fewest products that takes it
//
// call: forward, or any of i (input's gradient), g and u (the weights').  Every
// matrix has rows of `pad` elements more than it is wide.  A kernel is named by its
// template arguments as in the library's symbols.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>
#include <random>
#include <set>
#include <string>

#include "step_stub.h"

using namespace ptored::step;

namespace {

void* fake(int k) { return reinterpret_cast<void*>((uintptr_t)(k + 1) << 38); }

struct Case {
    int dtype;
    long long rows, cols, wide, pad;
    std::string call;
};

std::string text(const char* format, ...) {
    char line[160];
    va_list args;
    va_start(args, format);
    std::vsnprintf(line, sizeof line, format, args);
    va_end(args);
    return line;
}

// The kernel of a product that is launched alone.
std::string kernel_of(const Product& p) {
    const ProductArgs& a = p.a;
    if (a.shape >= kFew16) {
        bool odd = false;
        if (a.shape == kFew16 && p.dtype != PTORED_F32) {
            int64_t at = (int64_t)(uintptr_t)a.a[0] | (a.m > 1 ? a.a_ld[0] : 0);
            for (int i = 0; i < 2; ++i) at |= (int64_t)(uintptr_t)a.b[i] | a.b_ld[i];
            odd = at & 2;
        }
        const char* blocks = a.shape == kFew16 ? "1, 1, 4" : a.shape == kFew32 ? "1, 2, 4" : "2, 4, 2";
        return text("few_kernel<%d, %d, %s, %s>", p.dtype, odd ? 8 : a.waves, blocks, odd ? "true" : "false");
    }
    const char* tile = nullptr;
    const bool many = p.kind != kWeight;
    switch (a.shape) {
        case kTile128: tile = a.direct ? "2, 2, 2, 2, 128, 2, 0" : many ? "4, 2, 1, 2, 128, 2, 1" : "2, 2, 2, 2, 128, 2, 1"; break;
        case kTile128Deep: tile = "4, 2, 1, 2, 128, 4, 0"; break;
        case kTile256: tile = a.direct ? "2, 4, 4, 2, 128, 2, 0" : "2, 4, 4, 2, 128, 2, 1"; break;
        case kTile64: tile = "2, 1, 1, 2, 128, 8, 0"; break;
        case kTile128x32: tile = "4, 1, 1, 2, 128, 6, 0"; break;
        case kTile32x128: tile = a.direct ? "1, 4, 1, 1, 128, 4, 0" : "1, 4, 1, 1, 128, 2, 1"; break;
        case kTile64x128: tile = a.direct ? "2, 2, 1, 2, 128, 3, 0" : "2, 2, 1, 2, 128, 2, 1"; break;
        case kTileSplit: tile = "4, 2, 2, 2, 128, 2, 2"; break;
        default: tile = "2, 2, 2, 2, 128, 2, 3";
    }
    return text("product_kernel<%d, %d, %s>", p.dtype, p.kind, tile);
}

// The kernels that a call launches; empty if it is refused.
std::set<std::string> kernels_of(const Case& c) {
    const ptored_ffn_params p{c.rows, c.cols, c.wide, c.dtype, 0};
    const int64_t D = c.cols + c.pad, F = c.wide + c.pad, room = int64_t(1) << 37;
    auto mat = [](int k, int64_t ld) { return ptored_rows{fake(k), ld}; };
    g_seen = {};
    int st;
    if (c.call == "forward") {
        st = ptored_gated_ffn(&p, mat(1, D), mat(2, D), mat(3, D), mat(4, F), mat(5, F), mat(6, F), fake(12), room,
                              nullptr);
    } else {
        auto has = [&](char k) { return c.call.find(k) != std::string::npos; };
        ptored_ffn_grad_io io{};
        io.dy = mat(1, F);
        io.gate = mat(2, F);
        io.up = mat(3, F);
        io.dgate = mat(4, F);
        io.dup = mat(5, F);
        io.x = mat(6, D);
        io.w_gate = mat(7, D);
        io.w_up = mat(8, D);
        if (has('i')) io.dx = mat(9, D);
        if (has('g')) io.dw_gate = mat(10, D);
        if (has('u')) io.dw_up = mat(11, D);
        io.dw_dtype = c.dtype;
        io.workspace = fake(12);
        io.workspace_bytes = room;
        st = ptored_gated_ffn_backward(&p, &io, nullptr);
    }
    std::set<std::string> out;
    if (st != PTORED_OK) return out;
    const auto& seen = g_seen.products;
    if (!g_seen.firsts.empty()) {
        const ProductArgs &w = seen[0].a, &d = seen[1].a;
        out.insert(text("product_both_kernel<%d, %d>", c.dtype, w.direct && d.direct ? 0 : 1));
        if (w.splits > 1 && d.splits > 1) {
            out.insert(text("product_both_join_kernel<%d>", c.dtype));
            return out;
        }
    }
    for (const Product& q : seen) {
        if (g_seen.firsts.empty()) out.insert(kernel_of(q));
        if (q.a.splits > 1) out.insert(text("product_join_kernel<%d, %d>", q.dtype, q.kind));
    }
    return out;
}

std::string line_of(const Case& c) {
    return text("%d %lld %lld %lld %lld %s", c.dtype, c.rows, c.cols, c.wide, c.pad, c.call.c_str());
}

}  // namespace

int main(int argc, char** argv) {
    if (argc == 2 && std::strcmp(argv[1], "cases") == 0) {
        Case c;
        char call[16];
        while (std::scanf("%d %lld %lld %lld %lld %15s", &c.dtype, &c.rows, &c.cols, &c.wide, &c.pad, call) == 6) {
            c.call = call;
            std::string line;
            for (const std::string& k : kernels_of(c)) line += (line.empty() ? "" : "; ") + k;
            std::printf("%s\n", line.c_str());
        }
        return 0;
    }
    if (argc != 3 || std::strcmp(argv[1], "all") != 0) return 2;
    std::mt19937_64 rng(7);
    auto size = [&](double most) {
        const double u = std::uniform_real_distribution<double>(0, 1)(rng);
        const long long n = (long long)(std::pow(most, u) + 0.5);
        const int kind = (int)(rng() % 3);
        return std::max<long long>(1, kind == 0 ? n / 64 * 64 : kind == 1 ? n / 8 * 8 : n);
    };
    std::map<std::string, std::pair<double, Case>> found;
    const char* calls[] = {"forward", "i", "g", "u", "gu", "ig", "iu", "igu"};
    for (long long i = std::atoll(argv[2]); i > 0; --i) {
        Case c;
        c.dtype = (int)(rng() % 3);
        c.rows = size(16384);
        c.cols = size(16384);
        c.wide = size(16384);
        c.pad = (long long)(rng() % 4) * (rng() % 2 ? 1 : 8);
        c.call = calls[rng() % 2 ? 0 : rng() % 8];
        const double work = (double)c.rows * (double)c.cols * (double)c.wide;
        for (const std::string& k : kernels_of(c)) {
            const auto at = found.find(k);
            if (at == found.end() || work < at->second.first) found[k] = {work, c};
        }
    }
    for (const auto& f : found) std::printf("%s | %s\n", f.first.c_str(), line_of(f.second.second).c_str());
    return 0;
}
