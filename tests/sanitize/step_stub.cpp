// step_stub.cpp -- test-only stand-ins for the kernel launches of the step's
// operators, so that their host code (argument checks, tiles and splits, tables of
// gradients) runs on a machine without a GPU.  Nothing is launched;
// tests/sanitize/step_launches.cpp looks at what launches would have been handed.
#include "step_stub.h"

namespace ptored {
namespace step {

Launches g_seen;

#define PTORED_PRODUCT(kind_, name, T, dt)                 \
    int product_##name##_##T(const ProductArgs& a, hipStream_t) { \
        g_seen.products.push_back({kind_, dt, a});         \
        return kOk;                                        \
    }
#define PTORED_STUBS(T, dt)                                                              \
    int layer_norm_##T(const LayerNormArgs&, hipStream_t) { return ++g_seen.others, kOk; } \
    int layer_grad_##T(const LayerGradArgs& a, hipStream_t) {                            \
        g_seen.layers.push_back(a);                                                      \
        return kOk;                                                                      \
    }                                                                                    \
    PTORED_PRODUCT(kForward, forward, T, dt)                                             \
    PTORED_PRODUCT(kInput, input, T, dt)                                                 \
    PTORED_PRODUCT(kWeight, weight, T, dt)                                               \
    int product_both_##T(const ProductPair& p, hipStream_t) {                            \
        g_seen.products.push_back({kWeight, dt, p.weight});                              \
        g_seen.products.push_back({kInput, dt, p.input});                                \
        g_seen.firsts.push_back(p.first);                                                \
        return kOk;                                                                      \
    }                                                                                    \
    int product_slope_##T(const SlopeArgs&, hipStream_t) { return ++g_seen.others, kOk; }
PTORED_STUBS(f32, PTORED_F32)
PTORED_STUBS(bf16, PTORED_BF16)
PTORED_STUBS(f16, PTORED_F16)

int grad_table(const GradPack& a, hipStream_t) { return g_seen.packs.push_back(a), kOk; }
int grad_sums(const GradList& a, hipStream_t) { return g_seen.sums.push_back(a), kOk; }
int grad_join(const GradList& a, hipStream_t) { return g_seen.joins.push_back(a), kOk; }
int grad_scale(const GradList& a, hipStream_t) { return g_seen.scales.push_back(a), kOk; }

}  // namespace step
}  // namespace ptored
