// gate_select.hpp — the rule of one gated choice of experts and its order
// keys. Internal to libmoe_fp8.so.
#pragma once

#include "device.hpp"

namespace moe {

constexpr int kMaxGroups = 64;  // a group's score is made by at least one lane
// four tokens a workgroup of 256 threads, fewer than 2^32 threads a grid
constexpr int64_t kMaxGateTokens = ((int64_t)1 << 26) - 4;
constexpr float kMaskedLogit = -3.3e38f;  // at or below: the expert is masked

// moe_gating, checked and completed for one layer.
struct GateRule {
  int experts, top_k;
  int groups, per_group, top_groups, rank;
  int nv;               // experts per lane, consecutive ones
  bool vec;             // a lane's logits can be read with vector loads
  bool fast;            // every lane lies in one group: fp32 keys first
  int group_lanes;      // (fast) lanes of a group, and one over it
  float inv_group_lanes;
  bool softmax, renorm;
  float scale;
};

// fp64 values as unsigned keys in the same order (-0 as +0; no NaN comes
// here). Every value's key is above the two marks.
constexpr uint64_t kKeyAbsent = 0, kKeyMasked = 1;
__device__ __forceinline__ uint64_t order_key(double c) {
  const uint64_t b = (uint64_t)__double_as_longlong(c + 0.0);
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double key_value(uint64_t k) {
  return __longlong_as_double((long long)((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}
__device__ __forceinline__ uint64_t readlane_u64(uint64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return ((uint64_t)hi << 32) | lo;
}

}  // namespace moe
