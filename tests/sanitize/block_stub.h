// block_stub.h -- what tests/sanitize/block_stub.cpp records of a call.
#pragma once

#include "block/block_plan.h"

namespace ptored {
namespace block {

struct Launches {
    int count;  // since the program began
    GradArgs grad;
    WgradArgs wgrad;
};
extern Launches g_last;

}  // namespace block
}  // namespace ptored
