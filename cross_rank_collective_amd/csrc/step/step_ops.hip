// step_ops.hip -- kernel instances of the step's operators for one element
// type; built once per type with -DPTORED_INST_DT=<a ptored_dtype name>
// -DPTORED_INST_NAME=<its suffix>.
#include "layer_norm.hpp"
#include "product.hpp"

#if !defined(PTORED_INST_DT) || !defined(PTORED_INST_NAME)
#error "step_ops.hip needs -DPTORED_INST_DT=<ptored_dtype> -DPTORED_INST_NAME=<suffix>"
#endif

#define PTORED_JOIN2(a, b) a##b
#define PTORED_JOIN(a, b) PTORED_JOIN2(a, b)
#define PTORED_NAMED(f) PTORED_JOIN(f, PTORED_INST_NAME)

namespace ptored {
namespace step {

int PTORED_NAMED(layer_norm_)(const LayerNormArgs& a, hipStream_t s) {
    return layer_norm_launch<PTORED_INST_DT>(a, s);
}
int PTORED_NAMED(layer_grad_)(const LayerGradArgs& a, hipStream_t s) {
    return layer_grad_launch<PTORED_INST_DT>(a, s);
}
int PTORED_NAMED(product_forward_)(const ProductArgs& a, hipStream_t s) {
    return product_launch<PTORED_INST_DT, kForward>(a, s);
}
int PTORED_NAMED(product_input_)(const ProductArgs& a, hipStream_t s) {
    return product_launch<PTORED_INST_DT, kInput>(a, s);
}
int PTORED_NAMED(product_weight_)(const ProductArgs& a, hipStream_t s) {
    return product_launch<PTORED_INST_DT, kWeight>(a, s);
}
int PTORED_NAMED(product_both_)(const ProductPair& p, hipStream_t s) {
    return product_both_launch<PTORED_INST_DT>(p, s);
}
int PTORED_NAMED(product_slope_)(const SlopeArgs& a, hipStream_t s) {
    return slope_launch<PTORED_INST_DT>(a, s);
}

}  // namespace step
}  // namespace ptored
