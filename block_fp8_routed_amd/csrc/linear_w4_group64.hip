// linear_w4_group64.hip — the 4-bit products with groups of 64 columns (a file of its own
// so that the group sizes compile side by side).
#include "linear_w4.hpp"

namespace moe {

void launch_w4_group64(const W4Args& p, void* workspace, hipStream_t s) {
  launch_w4_group<64>(p, workspace, s);
}

}  // namespace moe
