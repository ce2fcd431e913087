// block_ops.hip -- kernel instances of the block-boundary operators for one
// element type; built once per type with -DPTORED_INST_DT=<a ptored_dtype
// name> -DPTORED_INST_NAME=<its suffix>.
#include "block_norm.hpp"
#include "block_norm_backward.hpp"
#include "checkpoint.hpp"
#include "checkpoint_wgrad.hpp"

#if !defined(PTORED_INST_DT) || !defined(PTORED_INST_NAME)
#error "block_ops.hip needs -DPTORED_INST_DT=<ptored_dtype> -DPTORED_INST_NAME=<suffix>"
#endif

#define PTORED_JOIN2(a, b) a##b
#define PTORED_JOIN(a, b) PTORED_JOIN2(a, b)
#define PTORED_NAMED(f) PTORED_JOIN(f, PTORED_INST_NAME)

namespace ptored {
namespace block {

int PTORED_NAMED(norm_)(const NormArgs& a, hipStream_t s) {
    return norm_launch<PTORED_INST_DT>(a, s);
}
int PTORED_NAMED(grad_)(const GradArgs& a, hipStream_t s) {
    return grad_launch<PTORED_INST_DT>(a, s);
}
int PTORED_NAMED(pack_)(const PackArgs& a, hipStream_t s) {
    return pack_launch<PTORED_INST_DT, true>(a, s);
}
int PTORED_NAMED(unpack_)(const PackArgs& a, hipStream_t s) {
    return pack_launch<PTORED_INST_DT, false>(a, s);
}
int PTORED_NAMED(wgrad_)(const WgradArgs& a, hipStream_t s) {
    return wgrad_launch<PTORED_INST_DT>(a, s);
}

}  // namespace block
}  // namespace ptored
