// block_launches.cpp -- drives the host code of the block-boundary operators
// through the C ABI with made-up device addresses, linked against
// tests/sanitize/block_stub.cpp instead of the kernels.  Built with
// AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_block_launches_cpu.py, which runs one check at a time (by name);
// needs no GPU.
#include <cstdint>
#include <cstdio>
#include <cstring>

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

}  // namespace

int main(int argc, char** argv) {
    const struct {
        const char* name;
        int (*check)();
    } checks[] = {{"no_gate", no_gate}, {"no_columns", no_columns}, {"eps_not_read", eps_not_read}};
    for (const auto& c : checks)
        if (argc == 2 && std::strcmp(argv[1], c.name) == 0) return c.check();
    std::printf("no such check\n");
    return 2;
}
