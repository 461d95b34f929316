// linear_w4_group32.hip — the 4-bit products with groups of 32 columns (a file of its own
// so that the group sizes compile side by side).
#include "linear_w4.hpp"

namespace moe {

void launch_w4_group32(const W4Args& p, void* workspace, hipStream_t s) {
  launch_w4_group<32>(p, workspace, s);
}

}  // namespace moe
