// step_stub.h -- what tests/sanitize/step_stub.cpp records of calls.
#pragma once

#include <vector>

#include "step/step_plan.h"

namespace ptored {
namespace step {

struct Product {
    int kind, dtype;
    ProductArgs a;
};
struct Launches {
    std::vector<Product> products;
    std::vector<int> firsts;  // of launches of both gradients: workgroups of the weights'
    std::vector<LayerGradArgs> layers;
    std::vector<GradPack> packs;
    std::vector<GradList> sums, joins, scales;
    int others = 0;
};
extern Launches g_seen;

}  // namespace step
}  // namespace ptored
