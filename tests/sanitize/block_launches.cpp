// block_launches.cpp -- drives the host code of the block-boundary operators
// through the C ABI with made-up device addresses, linked against
// tests/sanitize/block_stub.cpp instead of the kernels.  Built with
// AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_block_launches_cpu.py, which runs one check at a time (by name);
// needs no GPU.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

#include "block_stub.h"

using namespace ptored::block;

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

// A backward call that wants everything, with a gate of `gate_rows` rows (0: none).
struct Call {
    ptored_block_params p{};
    ptored_block_grad_io io{};
    Call(int64_t rows, int64_t cols, int64_t gate_rows, int dtype) {
        p.rows = rows;
        p.cols = cols;
        p.post_weight = fake(1);
        p.pre_weight = fake(2);
        if (gate_rows > 0) p.gate = mat(3, cols);
        p.gate_rows = gate_rows;
        p.branch_scale = p.residual_scale = 1.0f;
        p.eps = 1e-6f;
        p.dtype = dtype;
        io.dz = mat(4, cols);
        io.dx_out = mat(5, cols);
        io.x_out = mat(6, cols);
        io.h = mat(7, cols);
        io.post_rstd = static_cast<float*>(fake(8));
        io.pre_rstd = static_cast<float*>(fake(9));
        io.dx = mat(10, cols);
        io.dh = mat(11, cols);
        if (gate_rows > 0) io.dgate = mat(12, cols);
        io.dpost_weight = fake(13);
        io.dpre_weight = fake(14);
        io.workspace = fake(15);
        io.workspace_bytes = int64_t(1) << 35;
    }
    int run() { return ptored_block_norm_backward(&p, &io, nullptr); }
};

// Without a gate its row count is not read, whatever a caller left there.
int no_gate() {
    for (int64_t left : {int64_t(0), int64_t(1), int64_t(4), int64_t(3), int64_t(-1)}) {
        Call c(64, 256, 0, PTORED_BF16);
        c.p.gate_rows = left;
        EXPECT(c.run() == PTORED_OK, "gate_rows %lld", (long long)left);
        const GradArgs& a = g_last.grad;
        EXPECT(a.gate.p == nullptr && a.chunk_gates == kOneGate, "gate_rows %lld", (long long)left);
        EXPECT(a.gate_units == 0 && a.gate_rows == 0,
               "gate_rows %lld: the gate's rows would be read from address 0", (long long)left);
    }
    return 0;
}

// Rows without columns: nothing to do, whatever is asked for.
int no_columns() {
    for (int dtype : {PTORED_F32, PTORED_BF16, PTORED_F16})
        for (int64_t rows : {int64_t(0), int64_t(1), int64_t(8), int64_t(5000)})
            for (int64_t gate_rows : {int64_t(0), int64_t(1), rows}) {
                int64_t bytes = -1;
                EXPECT(ptored_block_norm_backward_workspace(rows, 0, gate_rows, &bytes) == PTORED_OK &&
                           bytes == 0,
                       "workspace of %lld rows", (long long)rows);
                Call c(rows, 0, gate_rows, dtype);
                const int before = g_last.count;
                EXPECT(c.run() == PTORED_OK && g_last.count == before, "%lld rows", (long long)rows);
            }
    return 0;
}

// The backward pass takes the norms' reciprocals, and does not read eps.
int eps_not_read() {
    for (float eps : {-1.0f, __builtin_nanf("")}) {
        Call c(64, 256, 2, PTORED_BF16);
        c.p.eps = eps;
        EXPECT(c.run() == PTORED_OK, "eps %g", (double)eps);
    }
    return 0;
}

// The rows of every chunk, walked as the kernel walks them: each row once,
// gate rows as the chunk's form takes them, and no more workspace needed than
// the query says, whatever is wanted of the sums.
int row_cuts_of(int64_t rows, int64_t cols, int64_t gate_rows, int dtype, int wanted) {
    char what[160];
    std::snprintf(what, sizeof what, "%lld x %lld, %lld gate rows, type %d, wanted %d", (long long)rows,
                  (long long)cols, (long long)gate_rows, dtype, wanted);
    Call c(rows, cols, gate_rows, dtype);
    if (!(wanted & 1)) c.io.dgate = {};
    if (!(wanted & 2)) c.io.dpost_weight = nullptr;
    if (!(wanted & 4)) c.io.dpre_weight = nullptr;
    const bool gated = c.io.dgate.data != nullptr;
    int64_t bytes = -1;
    EXPECT(ptored_block_norm_backward_workspace(rows, cols, gated ? gate_rows : 0, &bytes) == PTORED_OK,
           "%s", what);
    c.io.workspace_bytes = bytes;
    EXPECT(c.run() == PTORED_OK, "%s", what);
    const GradArgs& a = g_last.grad;
    EXPECT(a.chunks * a.ws_slots * a.ws_pitch * 4 <= bytes, "%s: workspace", what);
    EXPECT(a.chunks >= 1 && a.chunks < (1 << 22), "%s: %lld chunks", what, (long long)a.chunks);
    std::vector<char> seen(rows, 0), gate_seen(gate_rows > 0 ? gate_rows : 1, 0);
    for (int64_t chunk = 0; chunk < a.chunks; ++chunk) {
        const int64_t unit = chunk / a.chunks_per_unit, part = chunk - unit * a.chunks_per_unit;
        const int64_t begin = unit * a.unit_rows + part * a.chunk_first;
        const int64_t left = a.unit_rows - part * a.chunk_first;
        int64_t n = (left + a.row_step - 1) / a.row_step;
        if (n > a.chunk_rows) n = a.chunk_rows;
        EXPECT(n >= 1, "%s: chunk %lld has %lld rows", what, (long long)chunk, (long long)n);
        const bool gate = a.gate.p != nullptr;
        int64_t now = gate ? begin / a.rows_per_gate : 0;
        int64_t end = a.chunk_gates == kOneGate ? n
                      : a.row_step > 1          ? 1
                                                : (now + 1) * a.rows_per_gate - begin;
        for (int64_t i = 0; i < n; ++i) {
            const int64_t row = begin + i * a.row_step;
            EXPECT(row < rows && !seen[row], "%s: row %lld of chunk %lld", what, (long long)row,
                   (long long)chunk);
            seen[row] = 1;
            if (gate && i == end) {  // the next gate row
                now += a.row_step;
                end += a.row_step > 1 ? 1 : a.rows_per_gate;
            }
            EXPECT(!gate || now == row / a.rows_per_gate, "%s: gate row of row %lld", what, (long long)row);
            // a chunk that writes a gate row's gradient holds all of its rows
            if (a.gate_direct && (i + 1 == end || i + 1 == n)) {
                EXPECT(now < gate_rows && !gate_seen[now] && i + 1 == end, "%s: gate row %lld", what,
                       (long long)now);
                gate_seen[now] = 1;
            }
        }
        // the joining kernel's gate row of a chunk
        EXPECT(!a.gate_joined || chunk / a.chunks_per_unit == begin / a.rows_per_gate, "%s: chunk %lld", what,
               (long long)chunk);
    }
    for (int64_t r = 0; r < rows; ++r) EXPECT(seen[r], "%s: row %lld left out", what, (long long)r);
    for (int64_t g = 0; a.gate_direct && g < gate_rows; ++g)
        EXPECT(gate_seen[g], "%s: gate row %lld left out", what, (long long)g);
    return 0;
}

int row_cuts() {
    uint64_t state = 9;
    auto draw = [&](int64_t n) {  // 0 to n - 1
        state = state * 6364136223846793005u + 1442695040888963407u;
        return (int64_t)((state >> 33) % (uint64_t)n);
    };
    const int64_t widths[] = {1, 7, 8, 33, 512, 513, 1023, 2048, 4096, 4097, 8192, 8193, 16384};
    for (int i = 0; i < 4000; ++i) {
        const int64_t cols = widths[draw(13)], per_gate = 1 + draw(draw(2) ? 12 : 700);
        const int64_t gates = draw(4) == 0 ? 0 : 1 + draw(draw(2) ? 12 : 600);
        const int64_t rows = gates == 0 ? 1 + draw(6000) : gates * per_gate;
        if (row_cuts_of(rows, cols, gates, (int)draw(3), (int)draw(8))) return 1;
    }
    return 0;
}

// The tokens of every split of a weight gradient: all of them, each once, and
// no more workspace needed than the query says.
int token_splits() {
    for (int dtype : {PTORED_F32, PTORED_BF16, PTORED_F16})
        for (int64_t rows : {1, 2, 31, 64, 127, 128, 129, 1001, 4096, 9001, 32768})
            for (int64_t outs : {1, 7, 8, 64, 129, 640, 2500})
                for (int64_t cols : {1, 15, 16, 65, 512, 2049}) {
                    int64_t bytes = -1;
                    EXPECT(ptored_checkpoint_wgrad_workspace(rows, outs, cols, dtype, &bytes) == PTORED_OK,
                           "query");
                    const int st = ptored_checkpoint_wgrad(
                        mat(1, outs), {fake(2), cols, fake(3), (cols + 31) / 32}, rows, outs, cols, dtype,
                        mat(4, cols), PTORED_F32, 0, fake(5), bytes, nullptr);
                    EXPECT(st == PTORED_OK, "%d", st);
                    const WgradArgs& a = g_last.wgrad;
                    EXPECT(a.splits >= 1 && (a.splits - 1) * a.rows_per_split < rows &&
                               a.splits * a.rows_per_split >= rows,
                           "%lld tokens, %d splits of %lld", (long long)rows, a.splits,
                           (long long)a.rows_per_split);
                    EXPECT(a.splits == 1 || a.splits * outs * a.ws_ld * 4 <= bytes, "workspace");
                    const int64_t tm = a.shape == kWgradWide ? 256 : 128;
                    const int64_t tn = a.shape == kWgradWide || (dtype == PTORED_F32 && a.shape == kWgradTile)
                                           ? 256
                                           : 128;
                    EXPECT(a.tiles_m * tm >= outs && (a.tiles_m - 1) * tm < outs, "tiles");
                    EXPECT(a.tiles_n * tn >= cols && (a.tiles_n - 1) * tn < cols, "tiles");
                    EXPECT(a.shape == kWgradFew || (outs >= 8 && cols >= 16), "rows shorter than a chunk");
                }
    return 0;
}

// A single row has no pitch: an output is an input's row whatever their pitches.
int one_row() {
    for (int64_t rows : {int64_t(1), int64_t(2)}) {
        const int want = rows == 1 ? PTORED_OK : PTORED_ERR_OVERLAP;
        Call c(rows, 256, 0, PTORED_BF16);
        c.io.dx = {c.io.dz.data, 512};
        EXPECT(c.run() == want, "backward, %lld rows", (long long)rows);
        ptored_block_io io{};
        io.x = mat(4, 256);
        io.x_out = mat(4, 1024);
        io.z = mat(5, 256);
        const void* parts[] = {fake(6), fake(5)};
        const int st = ptored_block_norm(parts, 2, 512, &c.p, &io, nullptr);
        EXPECT(st == want, "forward, %lld rows: %d", (long long)rows, st);
    }
    return 0;
}

}  // namespace

int main(int argc, char** argv) {
    const struct {
        const char* name;
        int (*check)();
    } checks[] = {{"no_gate", no_gate}, {"no_columns", no_columns}, {"eps_not_read", eps_not_read},
                {"row_cuts", row_cuts}, {"token_splits", token_splits}, {"one_row", one_row}};
    for (const auto& c : checks)
        if (argc == 2 && std::strcmp(argv[1], c.name) == 0) return c.check();
    std::printf("no such check\n");
    return 2;
}
