// block_stub.cpp -- test-only stand-ins for the kernel launches of the
// block-boundary operators, so that their host code (argument checks, row
// cuts, workspace needs) runs on a machine without a GPU.  Nothing is
// launched; tests/sanitize/block_launches.cpp looks at what a launch would
// have been handed.
#include "block_stub.h"

namespace ptored {
namespace block {

Launches g_last;

#define PTORED_STUBS(T)                                                              \
    int norm_##T(const NormArgs&, hipStream_t) { return ++g_last.count, kOk; }       \
    int grad_##T(const GradArgs& a, hipStream_t) {                                   \
        g_last.grad = a;                                                             \
        return ++g_last.count, kOk;                                                  \
    }                                                                                \
    int pack_##T(const PackArgs&, hipStream_t) { return ++g_last.count, kOk; }       \
    int unpack_##T(const PackArgs&, hipStream_t) { return ++g_last.count, kOk; }     \
    int wgrad_##T(const WgradArgs& a, hipStream_t) {                                 \
        g_last.wgrad = a;                                                            \
        return ++g_last.count, kOk;                                                  \
    }
PTORED_STUBS(f32)
PTORED_STUBS(bf16)
PTORED_STUBS(f16)

}  // namespace block
}  // namespace ptored
