// gate_select.hip — choice of experts with scores, a balance bias and groups
// (moe_select_experts, and the selection of moe_route_gated and
// moe_forward_gated).
//
// For one token with logits l over E experts in G equal groups:
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e))       score
//   c_e = s_e + b_e                                 what the choice goes by
//   a group's score is the sum of its r largest c, r = 1 or 2
//   S   = the k largest c among the experts of the top_groups best groups
//   g_j = s_{S_j} [/ sum_i s_{S_i}] * scale         gates
// Ties go to the lower expert (group) index, slots descend in c.
//
// Two experts' c often lie closer than fp32 tells apart (sigmoid scores of a
// 4096-token prompt over 512 experts hold several pairs within 1e-7 at the
// k-th place), so scores, c and their order are kept in fp64: MI355X runs an
// fp64 instruction at the rate of an fp32 one, and the gates' sums cost
// nothing more for it.
//
// A masked expert (logit NaN or not above -3.3e38, which takes -inf and the
// lowest finite value of fp32 and bf16) has score 0, adds nothing to its
// group and is chosen only when the kept groups run out of others (then the
// lowest index first, gate 0).
//
// One wavefront per token; lane L owns experts L, L + 64, ...
#include <cmath>

#include "gate_select.hpp"
#include "layer.hpp"

namespace moe {

// Logits of a caller's matrix, rows ld apart.
template <bool BF16>
struct MatrixLogits {
  const void* p;
  int64_t ld;
  template <int NV>
  __device__ __forceinline__ void load(float (&v)[NV], int64_t t, int E) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e0 = (threadIdx.x & 63) + 64 * i, e = e0 < E ? e0 : E - 1;
      if (BF16)
        v[i] = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[t * ld + e] << 16);
      else
        v[i] = reinterpret_cast<const float*>(p)[t * ld + e];
    }
  }
};

// The router's partial logits per slice of H, summed in slice order, plus the
// router's bias.
struct SliceLogits {
  const float* p;
  int slices;
  int64_t T;
  const float* bias;
  float* out;  // may be null: the finished logits
  template <int NV>
  __device__ __forceinline__ void load(float (&v)[NV], int64_t t, int E) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e0 = (threadIdx.x & 63) + 64 * i, e = e0 < E ? e0 : E - 1;
      float a = p[t * E + e];
      for (int s = 1; s < slices; ++s) a += p[((size_t)s * T + t) * E + e];
      if (bias) a += bias[e];
      if (out && e0 < E) out[t * E + e] = a;
      v[i] = a;
    }
  }
};

template <int NV, class Logits>
__global__ __launch_bounds__(256) void gate_select_kernel(Logits lg,
                                                         const float* __restrict__ balance,
                                                         GateRule r, int64_t T,
                                                         int32_t* __restrict__ topk,
                                                         float* __restrict__ gates,
                                                         int32_t* __restrict__ zero_word) {
  __shared__ double sc_lds[4][64 * NV];
  __shared__ double c_lds[4][64 * NV];
  if (zero_word && blockIdx.x == 0 && threadIdx.x == 0) *zero_word = 0;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= T) return;  // (no workgroup barrier follows)
  const int E = r.experts;
  float v[NV];
  lg.template load<NV>(v, t, E);
  double sc[NV];
  bool ok[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) ok[i] = lane + 64 * i < E && v[i] > kMaskedLogit;
  if (r.softmax) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = fminf(v[i], 3.402823466e38f);  // +inf shares the mass as the largest value
      if (ok[i]) m = fmaxf(m, v[i]);
    }
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      sc[i] = ok[i] ? exp((double)v[i] - (double)m) : 0.0;
      z += sc[i];
    }
    for (int o = 32; o; o >>= 1) z += __shfl_xor(z, o);
#pragma unroll
    for (int i = 0; i < NV; ++i) sc[i] = z > 0.0 ? sc[i] / z : 0.0;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) sc[i] = ok[i] ? 1.0 / (1.0 + exp(-(double)v[i])) : 0.0;
  }
  uint64_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 64 * i;
    const double c = sc[i] + (balance && e < E ? (double)balance[e] : 0.0);
    key[i] = e < E ? (ok[i] ? order_key(c) : kKeyMasked) : kKeyAbsent;
    sc_lds[wave][e] = sc[i];
    c_lds[wave][e] = ok[i] ? c : -INFINITY;
  }
  // the wavefront's own LDS traffic is in order; the fence keeps the compiler to it
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (r.groups > 1) {
    const int lpg = r.lanes_per_group, g = lane / lpg, sub = lane & (lpg - 1);
    double a = -INFINITY, b = -INFINITY;  // the two largest c seen
    if (g < r.groups)
      for (int j = sub; j < r.per_group; j += lpg) {
        const double c = c_lds[wave][g * r.per_group + j];
        b = fmax(b, fmin(a, c));
        a = fmax(a, c);
      }
    for (int o = 1; o < lpg; o <<= 1) {
      const double a2 = __shfl_xor(a, o), b2 = __shfl_xor(b, o);
      b = fmax(fmax(b, b2), fmin(a, a2));
      a = fmax(a, a2);
    }
    const double gs = r.rank > 1 && b > -INFINITY ? a + b : a;
    const uint64_t gk = g < r.groups ? (a > -INFINITY ? order_key(gs) : kKeyMasked) : kKeyAbsent;
    int before = 0;  // groups that come before this lane's
    for (int j = 0; j < r.groups; ++j) {
      const uint64_t o = readlane_u64(gk, j * lpg);
      before += o > gk || (o == gk && j < g) ? 1 : 0;
    }
    const unsigned long long kept = __ballot(before < r.top_groups);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      const int eg = e < E ? e / r.per_group : 0;
      if (!((kept >> (eg * lpg)) & 1)) key[i] = kKeyAbsent;
    }
  }
  int mine = 0;
  for (int j = 0; j < r.top_k; ++j) {
    uint64_t lm = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) lm = key[i] > lm ? key[i] : lm;
    const uint64_t m = wave_max_u64(lm);
    uint32_t loc = 0xffffffffu;  // the lane's lowest expert holding the maximum
#pragma unroll
    for (int i = NV - 1; i >= 0; --i) loc = key[i] == m ? (uint32_t)(64 * i + lane) : loc;
    const int win = (int)~wave_max_u32(~loc);
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = win == 64 * i + lane ? kKeyAbsent : key[i];
    if (lane == j) mine = win;
  }
  double s = lane < r.top_k ? sc_lds[wave][mine] : 0.0;
  double den = 1.0;
  if (r.renorm) {
    den = s;
    for (int o = 8; o; o >>= 1) den += __shfl_xor(den, o, 16);
  }
  if (lane < r.top_k) {
    topk[t * r.top_k + lane] = mine;
    gates[t * r.top_k + lane] = (float)(den > 0.0 ? s / den * (double)r.scale : 0.0);
  }
}

template <class Logits>
static hipError_t launch(const Logits& lg, const float* balance, const GateRule& r, int64_t T,
                         int32_t* topk, float* gates, int32_t* zero_word, hipStream_t s) {
  const dim3 grid((unsigned)((T + 3) / 4));
  const int nv = (r.experts + 63) / 64;
#define MOE_GATE(NV) \
  gate_select_kernel<NV><<<grid, 256, 0, s>>>(lg, balance, r, T, topk, gates, zero_word)
  if (nv <= 1)
    MOE_GATE(1);
  else if (nv <= 2)
    MOE_GATE(2);
  else if (nv <= 4)
    MOE_GATE(4);
  else if (nv <= 8)
    MOE_GATE(8);
  else
    MOE_GATE(16);
#undef MOE_GATE
  return hipGetLastError();
}

moe_status gate_rule(const moe_gating* g, int experts, int top_k, GateRule* r) {
  if (!g) return MOE_ERR_NULL;
  if (g->score != MOE_SCORE_SOFTMAX && g->score != MOE_SCORE_SIGMOID) return MOE_ERR_SHAPE;
  if (g->renormalise != 0 && g->renormalise != 1) return MOE_ERR_SHAPE;
  if (!std::isfinite(g->scale)) return MOE_ERR_SHAPE;
  if (g->groups < 1 || experts % g->groups != 0) return MOE_ERR_SHAPE;
  const int per = experts / g->groups;
  if (g->top_groups < 1 || g->top_groups > g->groups) return MOE_ERR_SHAPE;
  if (g->group_rank < 1 || g->group_rank > 2) return MOE_ERR_SHAPE;
  if (g->groups > 1 && g->group_rank > per) return MOE_ERR_SHAPE;
  if (top_k > (int64_t)g->top_groups * per) return MOE_ERR_SHAPE;
  if (g->groups > kMaxGroups) return MOE_ERR_UNSUPPORTED;
  r->experts = experts;
  r->top_k = top_k;
  r->groups = g->groups;
  r->per_group = per;
  r->top_groups = g->top_groups;
  r->rank = g->group_rank;
  r->lanes_per_group = 1;
  while (2 * r->lanes_per_group * g->groups <= 64) r->lanes_per_group *= 2;
  r->softmax = g->score == MOE_SCORE_SOFTMAX;
  r->renorm = g->renormalise;
  r->scale = g->scale;
  return MOE_OK;
}

hipError_t launch_gate_select(const Dims& d, const GateRule& r, const float* plog,
                              const float* router_bias, const float* balance, int32_t* topk,
                              float* gates, float* logits_out, int32_t* zero_word,
                              hipStream_t s) {
  return launch(SliceLogits{plog, router_slices(d), d.T, router_bias, logits_out}, balance, r,
                d.T, topk, gates, zero_word, s);
}

}  // namespace moe

extern "C" moe_status moe_select_experts(const void* logits, moe_dtype dtype, int64_t ld,
                                         const float* balance_bias, const moe_gating* gating,
                                         int64_t tokens, int32_t experts, int32_t top_k,
                                         int32_t* topk_idx, float* gates, void* stream) {
  using namespace moe;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_SHAPE;
  if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts || ld < experts)
    return MOE_ERR_SHAPE;
  GateRule r;
  const moe_status st = gate_rule(gating, experts, top_k, &r);
  if (st != MOE_OK) return st;
  if (experts > kMaxExperts || top_k > kMaxTopK || tokens >= ((int64_t)1 << 32))
    return MOE_ERR_UNSUPPORTED;
  if (!logits || !topk_idx || !gates) return MOE_ERR_NULL;
  if (tokens == 0) return MOE_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e =
      dtype == MOE_BF16
          ? launch(MatrixLogits<true>{logits, ld}, balance_bias, r, tokens, topk_idx, gates,
                   nullptr, s)
          : launch(MatrixLogits<false>{logits, ld}, balance_bias, r, tokens, topk_idx, gates,
                   nullptr, s);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
