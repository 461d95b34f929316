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
// k-th place), so the choice is fp64's. Only close calls need fp64, though: a
// wavefront selects by fp32 keys whose error is bounded, draws on past top_k
// while the next key is close to the last one, and where a decision was close
// computes just the drawn experts' scores in fp64 (where it was the groups', those
// of all experts of the token). The gates are fp64 rounded once.
//
// A masked expert (logit NaN or not above -3.3e38, which takes -inf and the
// lowest finite value of fp32 and bf16) has score 0, adds nothing to its
// group and is chosen only when the kept groups run out of others (then the
// lowest index first, gate 0).
//
// A token takes LPT lanes. Lane L of it owns nv consecutive experts L nv, L nv + 1,
// ...: the lowest lane that holds a value then holds the lowest expert with
// it, and where nv divides the group size a lane lies in one group.
//
// Reading the logits is a tenth of the time. Where tokens share wavefronts the
// kernel's own instructions bound it (30001 tokens of 160 experts: 1400 a
// wavefront, 17 us of 22.8). A token of its own has 920 for 512 experts in groups,
// 6 us of the 15.4 of 4096 tokens; the rest is the chain of its draws, one after
// the other and each a row of cross-lane steps, which four wavefronts a SIMD do
// not hide. 1 token of 512 experts 5.5 us, 48 tokens of 128 experts 5.7.
#include <cmath>
#include <type_traits>

#include "gate_select.hpp"
#include "layer.hpp"

namespace moe {

// Logits of a caller's matrix, rows ld apart. load: the lane's experts e0 ..
// e0 + nv - 1 (what lies past nv or E is the row's first).
template <bool BF16>
struct MatrixLogits {
  static constexpr bool kBf16 = BF16;
  const void* p;
  int64_t ld;
  template <int NV>
  __device__ __forceinline__ void load(float (&v)[NV], int64_t t, const GateRule& r, int e0) const {
    if (BF16) {
      const uint16_t* row = reinterpret_cast<const uint16_t*>(p) + t * ld;
      if (NV >= 2 && r.vec) {  // nv = NV and every lane's experts aligned and whole
        const uint16_t* at = row + (e0 < r.experts ? e0 : 0);
        uint32_t w[(NV + 1) / 2];
#pragma unroll
        for (int i = 0; i < NV / 2; i += 4) {
          if constexpr (NV == 2) w[0] = *reinterpret_cast<const uint32_t*>(at);
          if constexpr (NV == 4) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(at);
          if constexpr (NV >= 8) *reinterpret_cast<uint4*>(w + i) = ld16(at + 2 * i);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
        return;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
        v[i] = __uint_as_float((uint32_t)row[e0 + i < r.experts && i < r.nv ? e0 + i : 0] << 16);
    } else {
      const float* row = reinterpret_cast<const float*>(p) + t * ld;
      if (NV >= 2 && r.vec) {
        const float* at = row + (e0 < r.experts ? e0 : 0);
        if constexpr (NV == 2)
          *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(at);
        else
#pragma unroll
          for (int i = 0; i + 3 < NV; i += 4)
            *reinterpret_cast<float4*>(v + i) = *reinterpret_cast<const float4*>(at + i);
        return;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = row[e0 + i < r.experts && i < r.nv ? e0 + i : 0];
    }
  }
};

// The router's partial logits per slice of H, summed in slice order, plus the
// router's bias.
struct SliceLogits {
  static constexpr bool kBf16 = false;
  const float* p;
  int slices;
  int64_t T;
  const float* bias;
  float* out;  // may be null: the finished logits
  template <int NV>
  __device__ __forceinline__ void load(float (&v)[NV], int64_t t, const GateRule& r, int e0) const {
    const int E = r.experts;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = 0.f;
    for (int s = 0; s < slices; ++s)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float a = p[((size_t)s * T + t) * E + (e0 + i < E && i < r.nv ? e0 + i : 0)];
        v[i] = s ? v[i] + a : a;
      }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e0 + i < E && i < r.nv) {
        if (bias) v[i] += bias[e0 + i];
        if (out) out[t * E + e0 + i] = v[i];
      }
  }
};

// e^x in fp64 for x up to 710 (infinite from 709.78 on), within 2^-49: x = n ln 2
// + r, |r| <= 0.35, and the exponential series to r^12 (the rest is below 2^-50).
__device__ __forceinline__ double exp64(double x) {
  // ln 2 to 28 bits (n kLn2Hi is exact) and the rest
  constexpr double kLog2e = 0x1.71547652b82fep+0, kLn2Hi = 0x1.62e42fep-1,
                   kLn2Lo = 0x1.f473de6af278fp-30;
  x = fmax(x, -746.0);  // 0 from here down
  const double n = __builtin_rint(x * kLog2e);
  const double r = fma(-n, kLn2Lo, fma(-n, kLn2Hi, x));
  double p = 1.0 / 479001600.0;
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}
// Descending sort of N (a power of two) keys, odd-even merge network.
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int h = p; h >= 1; h /= 2)
#pragma unroll
      for (int j = h % p; j + h < N; j += 2 * h)
#pragma unroll
        for (int i = 0; i < h; ++i)
          if (i + j + h < N && (i + j) / (2 * p) == (i + j + h) / (2 * p)) {
            const uint32_t a = k[i + j], b = k[i + j + h];
            k[i + j] = max(a, b);
            k[i + j + h] = min(a, b);
          }
}

// ---- values across the LPT lanes (16 or 64) of a token ----
// Four DPP steps leave a 16-lane row's total in all its lanes; rows and halves
// of the wavefront then meet in gfx950's lane swaps: with both operands the
// same register, one result holds the even rows (the lower half) twice and the
// other the odd ones.
template <int LPT, class Op>
__device__ __forceinline__ uint32_t token_reduce(uint32_t v, Op op) {
  v = op(v, (uint32_t)dpp_i<kDppXor1>((int)v));
  v = op(v, (uint32_t)dpp_i<kDppXor2>((int)v));
  v = op(v, (uint32_t)dpp_i<kDppHalfMirror>((int)v));
  v = op(v, (uint32_t)dpp_i<kDppMirror>((int)v));
  if (LPT == 64) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op((uint32_t)r[0], (uint32_t)r[1]);
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op((uint32_t)h[0], (uint32_t)h[1]);
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t token_max(uint32_t v) {
  return token_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int LPT>
__device__ __forceinline__ float token_sum(float v) {
  return __uint_as_float(token_reduce<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ double make_f64(uint32_t lo, uint32_t hi) {
  return __longlong_as_double((long long)((uint64_t)hi << 32 | lo));
}
template <int LPT>
__device__ __forceinline__ double token_sum(double v) {
  const auto step = [&](auto ctrl) {
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    v += make_f64((uint32_t)dpp_i<decltype(ctrl)::value>((int)(uint32_t)b),
                  (uint32_t)dpp_i<decltype(ctrl)::value>((int)(b >> 32)));
  };
  step(std::integral_constant<int, kDppXor1>());
  step(std::integral_constant<int, kDppXor2>());
  step(std::integral_constant<int, kDppHalfMirror>());
  step(std::integral_constant<int, kDppMirror>());
  if (LPT == 64) {
    uint64_t b = (uint64_t)__double_as_longlong(v);
    auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
    auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false,
                                               false);
    v = make_f64(lo[0], hi[0]) + make_f64(lo[1], hi[1]);
    b = (uint64_t)__double_as_longlong(v);
    lo = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
    hi = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
    v = make_f64(lo[0], hi[0]) + make_f64(lo[1], hi[1]);
  }
  return v;
}
// the token's bits of a wavefront mask, at bit 0
template <int LPT>
__device__ __forceinline__ uint64_t token_bits(unsigned long long b, int base) {
  if (LPT == 64) return b;
  const uint32_t half = base & 32 ? (uint32_t)(b >> 32) : (uint32_t)b;
  return (half >> (base & 16)) & 0xffffu;
}
template <int LPT>
__device__ __forceinline__ int first_bit(uint64_t b) {
  return LPT == 64 ? __ffsll((unsigned long long)b) - 1 : __ffs((uint32_t)b) - 1;
}

// LDS of one wavefront. Expert i of lane L is at slot 64 i + L: lanes side by
// side, so that their reads and writes do not meet in a bank.
template <int NV, int LPT>
struct GateLds {
  float raw[64 * NV];     // logits, -inf for masked and absent experts
  uint64_t key[LPT * NV]; // exact choice of one token: order keys of c, by expert
  float head[2][64];      // each lane's two largest c
  alignas(16) float gs[64];  // groups' scores
  float2 edge[2][4];      // the last group kept and the first dropped: score, magnitude
  uint2 list[64];         // lane j of a token: the j-th key drawn and its slot
  double c[64];           // c of the drawn experts
};

// The softmax's sum of e^(l - top) over the token's lanes, nv logits each.
template <int LPT>
__device__ __forceinline__ double softmax_sum(int nv, const float* raw, float top) {
  double z = 0.0;
#pragma unroll 2
  for (int i = 0; i < nv; ++i) z += exp64((double)raw[64 * i] - (double)top);  // (-inf adds 0)
  return token_sum<LPT>(z);
}

// An expert's score from its logit (-inf: masked); softmax: not yet divided
// by the sum. A sigmoid is 0 where its exponential leaves fp64's range.
__device__ __forceinline__ double score64(const GateRule& r, float logit, float top) {
  const double x = r.softmax ? (double)logit - (double)top : fmin(-(double)logit, 710.0);
  const double e = exp64(x);
  const double s = r.softmax ? e : 1.0 / (1.0 + e);
  return logit > kMaskedLogit ? s : 0.0;
}

// ---- the exact choice, one token by the whole wavefront ----
// Rolled loops over LDS (few tokens come here). base: the token's first lane;
// lanes take every 64th expert.

// keys of c of all experts into lds.key
template <int NV, int LPT>
__device__ __forceinline__ void exact_keys(const GateRule& r, int base, float top,
                                           const float* __restrict__ balance, GateLds<NV, LPT>& lds) {
  const int lane = threadIdx.x & 63;
  double z = 1.0;
  if (r.softmax) {
    z = 0.0;
    for (int e = lane; e < r.experts; e += 64)
      z += exp64((double)lds.raw[64 * (e % r.nv) + base + e / r.nv] - (double)top);
    z = token_sum<64>(z);
  }
#pragma unroll 1
  for (int e = lane; e < r.experts; e += 64) {
    const float v = lds.raw[64 * (e % r.nv) + base + e / r.nv];
    double c = score64(r, v, top);
    if (r.softmax) c = z > 0.0 ? c / z : 0.0;
    if (balance) c += (double)balance[e];
    lds.key[e] = v > kMaskedLogit ? order_key(c) : kKeyMasked;
  }
  wave_lds_fence();
}

// the kept groups by lds.key, as a mask
template <int NV, int LPT>
__device__ __forceinline__ unsigned long long exact_groups(const GateRule& r, GateLds<NV, LPT>& lds) {
  const int lane = threadIdx.x & 63;
  uint64_t mine = 0;  // lane g: the key of group g's score
#pragma unroll 1
  for (int g = 0; g < r.groups; ++g) {
    uint64_t a = 0, b = 0;  // the group's two largest keys among the lane's experts
    for (int j = lane; j < r.per_group; j += 64) {
      const uint64_t c = lds.key[g * r.per_group + j];
      if (c > a) {
        b = a;
        a = c;
      } else if (c > b) {
        b = c;
      }
    }
    const uint64_t m = wave_max_u64(a);
    const int wl = __ffsll((unsigned long long)__ballot(a == m)) - 1;
    const uint64_t m2 = wave_max_u64(lane == wl ? b : a);
    uint64_t k = kKeyMasked;
    if (m > kKeyMasked)
      k = order_key(key_value(m) + (r.rank > 1 && m2 > kKeyMasked ? key_value(m2) : 0.0));
    if (lane == g) mine = k;
  }
  int before = 0;
  for (int j = 0; j < r.groups; ++j) {
    const uint64_t o = readlane_u64(mine, j);
    before += o > mine || (o == mine && j < lane) ? 1 : 0;
  }
  return __ballot(lane < r.groups && before < r.top_groups);
}

// the whole choice: slots into lds.list[base + j].y, j < top_k
template <int NV, int LPT>
__device__ __forceinline__ void choose_exact(const GateRule& r, int base, float top,
                                             const float* __restrict__ balance,
                                             GateLds<NV, LPT>& lds) {
  const int lane = threadIdx.x & 63;
  exact_keys<NV, LPT>(r, base, top, balance, lds);
  if (r.groups > 1) {
    const unsigned long long kept = exact_groups<NV, LPT>(r, lds);
    wave_lds_fence();
#pragma unroll 1
    for (int e = lane; e < r.experts; e += 64)
      if (!((kept >> (e / r.per_group)) & 1)) lds.key[e] = kKeyAbsent;
    wave_lds_fence();
  }
#pragma unroll 1
  for (int j = 0; j < r.top_k; ++j) {
    uint64_t best = 0;
    int at = 0;
    for (int e = lane; e < r.experts; e += 64) {
      const uint64_t c = lds.key[e];
      if (c > best) {
        best = c;
        at = e;
      }
    }
    const uint64_t m = wave_max_u64(best);
    // the lowest expert that holds it (largest complement)
    const int e = (int)~wave_max_u32(best == m ? ~(uint32_t)at : 0u);
    if (lane == 0) {
      lds.list[base + j].y = (uint32_t)(64 * (e % r.nv) + base + e / r.nv);
      lds.key[e] = kKeyAbsent;
    }
    wave_lds_fence();
  }
}

// fp32 values as unsigned keys in the same order (no NaN).
__device__ __forceinline__ uint32_t order32(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value32(uint32_t h) {
  return __uint_as_float(h ^ ((uint32_t)((int32_t)~h >> 31) | 0x80000000u));
}

// The choice by fp32 keys, made exact where they are close; slots into
// lds.list[base + j].y, j < top_k. False for a token where that is not possible
// (masked experts have to be chosen, or too many are too close to tell).
//   Without a bias, and where a group's score is its best expert's, the
// logits' own order is the order of c: keys are the logits. Two count as close
// if they differ by 2^-40 or less, or lie where the score hardly moves any more
// (sigmoid: above 20; softmax: 700 below the largest).
//   Otherwise keys are c in fp32. Its error eps: sigmoid below 2^-21 (the
// exponential's error times s (1 - s), the reciprocal, the sum); softmax below
// 2^-18 / z + 2^-22 (z a sum of up to 1024 fp32 exponentials; d e^-d <= 0.37
// bounds what the rounded l - top does).
//   A key's low bits hold the expert's place in its lane, so that a lane's keys
// can be sorted as plain numbers; what they displace (cut) counts as error too.
//   A token draws its largest key top_k times, and on while the next one is
// close to the last of these. If any two neighbours are close, the drawn ones
// (one per lane) are ranked by fp64 c and index.
template <int NV, int LPT>
__device__ __forceinline__ bool choose_fast(const GateRule& r, const float (&v)[NV], float top,
                                            const float (&bias)[NV],
                                            const float* __restrict__ balance,
                                            GateLds<NV, LPT>& lds) {
  constexpr int kLow = NV <= 1 ? 0 : NV <= 2 ? 1 : NV <= 4 ? 2 : NV <= 8 ? 3 : 4;
  constexpr uint32_t kPlace = (1u << kLow) - 1u;
  constexpr int kCandidates = LPT < 32 ? LPT : 32;
  const int lane = threadIdx.x & 63, tl = lane & (LPT - 1), base = lane - tl;
  const bool by_logit = !balance && (r.groups == 1 || r.rank == 1);
  uint32_t key[NV];
  float eps = 0.f;
  float c[NV];
  if (by_logit) {
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = v[i] + 0.0f;  // -0 as +0
  } else if (r.softmax) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      c[i] = __expf(v[i] - top);  // 0 for masked experts
      z += c[i];
    }
    z = token_sum<LPT>(z);
    const float q = z > 0.f ? 1.0f / z : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = fmaf(c[i], q, bias[i]);
    eps = 0x1p-18f * q + 0x1p-22f;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      c[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-v[i])) + bias[i];
    eps = 0x1p-21f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    key[i] = v[i] > kMaskedLogit ? (order32(c[i]) & ~kPlace) | (kPlace - i) : 0u;
  sort_desc(key);
  constexpr float kCut = 1.0f / (float)(1 << (22 - kLow));  // two keys' cuts, of their values
  // whether x >= y (values of cut keys) may be the wrong way round
  const auto close = [&](float x, float y) {
    if (by_logit) {
      const bool range = r.softmax ? top - x < 700.f : y < 20.f && x > -700.f;
      return !(x - y > 0x1p-40f && range);
    }
    return !(x - y > 2.0f * eps + kCut * fmaxf(fabsf(x), fabsf(y)));
  };
  if (r.groups > 1) {
    // (from c itself: the keys' cut would leave a group's score eight times less sure)
    float a = -INFINITY, b = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float x = v[i] > kMaskedLogit ? c[i] : -INFINITY;
      b = fmaxf(b, fminf(a, x));
      a = fmaxf(a, x);
    }
    lds.head[0][lane] = a;
    if constexpr (NV > 1) lds.head[1][lane] = b;
    wave_lds_fence();
    // lane g of the token: group g
    const int lg = r.group_lanes;
    a = b = -INFINITY;
    for (int j0 = 0; j0 < lg; j0 += 8) {  // eight lanes' values requested together
      float x[8], y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = base + tl * lg + j0 + j;
        x[j] = lds.head[0][at < 64 ? at : 63];
        if constexpr (NV > 1) y[j] = lds.head[1][at < 64 ? at : 63];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j0 + j >= lg) x[j] = -INFINITY;
        b = fmaxf(b, fminf(a, x[j]));
        a = fmaxf(a, x[j]);
        if constexpr (NV > 1) b = fmaxf(b, j0 + j < lg ? y[j] : -INFINITY);
      }
    }
    const bool in = tl < r.groups, two = r.rank > 1 && b > -INFINITY;
    const float gs = in ? a + (two ? b : 0.f) : -INFINITY;
    const float mag = (a > -INFINITY ? fabsf(a) : 0.f) + (two ? fabsf(b) : 0.f);
    lds.gs[lane] = gs;
    wave_lds_fence();
    int before = 0;
    for (int j0 = 0; j0 < r.groups; j0 += 4) {  // (lanes past the groups hold -inf)
      const float4 o = *reinterpret_cast<const float4*>(&lds.gs[base + j0]);
      before += o.x > gs || (o.x == gs && j0 < tl) ? 1 : 0;
      before += o.y > gs || (o.y == gs && j0 + 1 < tl) ? 1 : 0;
      before += o.z > gs || (o.z == gs && j0 + 2 < tl) ? 1 : 0;
      before += o.w > gs || (o.w == gs && j0 + 3 < tl) ? 1 : 0;
    }
    uint64_t kept = token_bits<LPT>(__ballot(in && before < r.top_groups), base);
    if (r.top_groups < r.groups) {
      if (in && before == r.top_groups - 1) lds.edge[0][base / 16] = make_float2(gs, mag);
      if (in && before == r.top_groups) lds.edge[1][base / 16] = make_float2(gs, mag);
      wave_lds_fence();
      const float2 k = lds.edge[0][base / 16], d = lds.edge[1][base / 16];
      const bool empty = k.x == -INFINITY && k.y == 0.f && d.y == 0.f;
      // Equal logits on both sides of the cut are equal scores, of which the
      // lower groups were kept. So may be other logits, above or below them, and
      // then those take part in the tie.
      bool tie = by_logit && k.x == d.x;
      if (__ballot(tie)) {
        const bool also = in && gs != k.x && close(fmaxf(gs, k.x), fminf(gs, k.x));
        tie = tie && token_bits<LPT>(__ballot(also), base) == 0;
      }
      const bool sure =
          empty || (k.x > -INFINITY &&
                    (by_logit ? tie || (k.x != d.x && !close(k.x, d.x))
                              : k.x - d.x > 4.0f * eps + 0x1p-22f * fmaxf(k.y, d.y)));
      unsigned long long todo = __ballot(!sure);
      while (todo) {
        const int at = (__ffsll(todo) - 1) & ~(LPT - 1);
        exact_keys<NV, LPT>(r, at, readlane_f(top, at), balance, lds);
        const unsigned long long exact = exact_groups<NV, LPT>(r, lds);
        if (base == at) kept = exact;
        todo &= LPT == 64 ? 0ull : ~(((1ull << (LPT & 63)) - 1ull) << at);
        wave_lds_fence();
      }
    }
    const int own = (int)(((float)tl + 0.5f) * r.inv_group_lanes);
    const bool mykept = own < r.groups && ((kept >> own) & 1);
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = mykept ? key[i] : 0u;
  }
  // the lane that holds the token's largest key m first draws it as the n-th
  const auto draw = [&](uint32_t h, uint32_t m, int n, bool on) {
    const int wl = first_bit<LPT>(token_bits<LPT>(__ballot(h == m), base));
    if (on && tl == wl) {
      lds.list[base + n] = make_uint2(m, 64u * (kPlace - (key[0] & kPlace)) + (uint32_t)lane);
#pragma unroll
      for (int i = 0; i + 1 < NV; ++i) key[i] = key[i + 1];
      key[NV - 1] = 0u;
    }
  };
  uint32_t m = 0;
  bool none = false;
  for (int j = 0; j < r.top_k; ++j) {
    const uint32_t h = key[0] >> kLow;
    m = token_max<LPT>(h);
    draw(h, m, j, true);
    if (j == 0) none = m == 0u;
  }
  // a token without any expert (a row of padding): the lowest groups are kept,
  // and the lowest experts chosen
  if (none && tl < r.top_k)
    lds.list[lane] = make_uint2(0u, (uint32_t)(64 * (tl % r.nv) + base + tl / r.nv));
  bool ok = m != 0u || none;
  const float last = value32(m << kLow);
  int n = r.top_k;
  for (;;) {
    const uint32_t h = key[0] >> kLow;
    m = token_max<LPT>(h);
    bool more = ok && m != 0u && close(last, value32(m << kLow));
    if (more && n == kCandidates) ok = more = false;
    if (!__ballot(more)) break;
    draw(h, m, n, more);
    n += more ? 1 : 0;
  }
  wave_lds_fence();
  // neighbours: far enough apart, or the same numbers (the lower index came first)
  const uint2 won = lds.list[lane], next = lds.list[lane < 63 ? lane + 1 : 63];
  const bool mine = ok && tl < n;
  const float lj = lds.raw[mine ? won.y : 0];
  const float ln = lds.raw[ok && tl + 1 < n ? next.y : 0];
  const bool unsure = ok && !none && tl + 1 < n && close(value32(won.x << kLow), value32(next.x << kLow)) &&
                      (balance || lj != ln);
  const bool rank = ok && !none && (n > r.top_k || token_bits<LPT>(__ballot(unsure), base) != 0);
  if (__ballot(rank)) {
    const int e = mine ? ((int)(won.y & 63u) - base) * r.nv + (int)(won.y >> 6) : 0;
    double cx = mine ? score64(r, lj, top) : 0.0;
    if (balance) {
      if (r.softmax) cx /= softmax_sum<LPT>(r.nv, lds.raw + lane, top);
      cx += (double)balance[e];
    }
    lds.c[lane] = cx;
    lds.list[lane].x = (uint32_t)e;
    wave_lds_fence();
    int before = 0;
    for (int j = 0; __ballot(rank && j < n); ++j) {
      const double o = lds.c[base + j];
      const int oe = (int)lds.list[base + j].x;
      before += j < n && (o > cx || (o == cx && oe < e)) ? 1 : 0;
    }
    wave_lds_fence();
    if (rank && mine) lds.list[base + before].y = won.y;
    wave_lds_fence();
  }
  return ok;
}

// LPT lanes per token: 64, or 16 where tokens fill the chip (launch).
template <int NV, int LPT, class Logits, bool BALANCE>
__global__ __launch_bounds__(256) void gate_select_kernel(Logits lg,
                                                         const float* __restrict__ balance_,
                                                         GateRule r, int64_t T,
                                                         int32_t* __restrict__ topk,
                                                         float* __restrict__ gates,
                                                         int32_t* __restrict__ zero_word) {
  __shared__ GateLds<NV, LPT> all[4];
  if (zero_word && blockIdx.x == 0 && threadIdx.x == 0) *zero_word = 0;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int tl = lane & (LPT - 1), base = lane - tl;
  const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * (64 / LPT);
  if (t0 >= T) return;  // (no workgroup barrier follows)
  // a token past the end repeats the last one and stores nothing
  const int64_t t = t0 + base / LPT < T ? t0 + base / LPT : T - 1;
  const bool there = t0 + base / LPT < T;
  GateLds<NV, LPT>& lds = all[wave];
  const float* balance = BALANCE ? balance_ : nullptr;
  const int e0 = tl * r.nv;
  float v[NV], bias[NV];
  lg.template load<NV>(v, t, r, e0);
#pragma unroll
  for (int i = 0; i < NV; ++i)
    bias[i] = BALANCE ? balance[e0 + i < r.experts && i < r.nv ? e0 + i : 0] : 0.f;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool ok = i < r.nv && e0 + i < r.experts && v[i] > kMaskedLogit;
    // +inf counts as the largest value
    v[i] = ok ? fminf(v[i], 3.402823466e38f) : -INFINITY;
    top = fmaxf(top, v[i]);
    lds.raw[64 * i + lane] = v[i];
  }
  // (a token without any expert left: not -inf, so that no difference is NaN)
  if (r.softmax) top = fmaxf(value32(token_max<LPT>(order32(top))), -3.402823466e38f);
  wave_lds_fence();
  const bool ok = r.fast && choose_fast<NV, LPT>(r, v, top, bias, balance, lds);
  for (unsigned long long todo = __ballot(!ok); todo;) {
    const int at = (__ffsll(todo) - 1) & ~(LPT - 1);
    choose_exact<NV, LPT>(r, at, readlane_f(top, at), balance, lds);
    todo &= LPT == 64 ? 0ull : ~(((1ull << (LPT & 63)) - 1ull) << at);
  }
  // gates
  const bool mine = tl < r.top_k;
  const int slot = mine ? (int)lds.list[lane].y : base;
  double s = mine ? score64(r, lds.raw[slot], top) : 0.0;
  double den = 1.0;
  if (r.renorm)
    den = token_sum<16>(s);  // (top_k <= 16)
  else if (r.softmax)
    den = softmax_sum<LPT>(r.nv, lds.raw + lane, top);
  if (mine && there) {
    topk[t * r.top_k + tl] = ((slot & 63) - base) * r.nv + (slot >> 6);
    gates[t * r.top_k + tl] = (float)(den > 0.0 ? s / den * (double)r.scale : 0.0);
  }
}

// Experts per lane where LPT lanes take a token: the fewest that cover all;
// with groups, of those that divide a group, if there is one up to 16 (else 0).
static int lane_experts(const GateRule& r, int lpt) {
  int nv = (r.experts + lpt - 1) / lpt;
  if (r.groups > 1)
    while (nv <= 16 && r.per_group % nv != 0) ++nv;
  return nv <= 16 && (r.groups == 1 || r.groups <= lpt) ? nv : 0;
}

template <class Logits>
static hipError_t launch(const Logits& lg, const float* balance, GateRule r, int64_t T,
                         int32_t* topk, float* gates, int32_t* zero_word, int align,
                         hipStream_t s) {
  // Four tokens share a wavefront, and its instructions, where there are enough
  // of them to fill the chip; before that a token's own way through is what
  // counts. Measured, 64 lanes a token against 16, us: bf16 softmax, 128
  // experts, top 8: 2048 tokens 6.0 / 6.6, 4096 7.1 / 6.6, 8192 9.7 / 7.2, 30001
  // 23.7 / 13.8; 160 experts in 8 groups, top 6: 4096 8.5 / 8.8, 30001 33.1 /
  // 23.4. Two tokens of 512 experts: 16384 38.2 / 39.2, so not there.
  const bool share = T >= 4096 && r.experts <= 256 && lane_experts(r, 16) != 0;
  const int lpt = share ? 16 : 64;
  r.nv = lane_experts(r, lpt);
  r.fast = r.nv != 0;
  if (!r.fast) r.nv = (r.experts + 63) / 64;
  r.group_lanes = r.per_group / r.nv;
  r.inv_group_lanes = 1.0f / (float)(r.group_lanes ? r.group_lanes : 1);
  const int nv = r.nv;
  const dim3 grid((unsigned)((T + 256 / lpt - 1) / (256 / lpt)));
  const int full = nv <= 1 && lpt == 64   ? 1
                   : nv <= 2 && lpt == 64 ? 2
                   : nv <= 4              ? 4
                   : nv <= 8              ? 8
                                          : 16;
  // vector loads: whole lanes, on the boundary that their reach asks for
  const int size = Logits::kBf16 ? 2 : 4, span = nv * size < 16 ? nv * size : 16;
  r.vec = nv == full && r.experts % nv == 0 && align % span == 0;
#define MOE_GATE(NV, LPT)                                                                     \
  balance ? gate_select_kernel<NV, LPT, Logits, true><<<grid, 256, 0, s>>>(                   \
                lg, balance, r, T, topk, gates, zero_word)                                    \
          : gate_select_kernel<NV, LPT, Logits, false><<<grid, 256, 0, s>>>(                  \
                lg, nullptr, r, T, topk, gates, zero_word)
  switch (100 * lpt + full) {
    case 6401: MOE_GATE(1, 64); break;
    case 6402: MOE_GATE(2, 64); break;
    case 6404: MOE_GATE(4, 64); break;
    case 6408: MOE_GATE(8, 64); break;
    case 6416: MOE_GATE(16, 64); break;
    case 1604: MOE_GATE(4, 16); break;
    case 1608: MOE_GATE(8, 16); break;
    default: MOE_GATE(16, 16);
  }
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
  r->softmax = g->score == MOE_SCORE_SOFTMAX;
  r->renorm = g->renormalise;
  r->scale = g->scale;
  return MOE_OK;
}

hipError_t launch_gate_select(const Dims& d, const GateRule& r, const float* plog,
                              const float* router_bias, const float* balance, int32_t* topk,
                              float* gates, float* logits_out, int32_t* zero_word,
                              hipStream_t s) {
  return launch(SliceLogits{plog, router_slices(d), d.T, router_bias, logits_out}, balance, r, d.T,
                topk, gates, zero_word, 1, s);
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
  if (experts > kMaxExperts || top_k > kMaxTopK || tokens > kMaxGateTokens)
    return MOE_ERR_UNSUPPORTED;
  if (!logits || !topk_idx || !gates) return MOE_ERR_NULL;
  if (tokens == 0) return MOE_OK;
  hipStream_t s = static_cast<hipStream_t>(stream);
  // the largest power of two, up to 16, that every row's address is a multiple of
  const int64_t size = dtype == MOE_BF16 ? 2 : 4;
  int align = 16;
  while (reinterpret_cast<uintptr_t>(logits) % align != 0 || ld * size % align != 0) align /= 2;
  const hipError_t e =
      dtype == MOE_BF16
          ? launch(MatrixLogits<true>{logits, ld}, balance_bias, r, tokens, topk_idx, gates,
                   nullptr, align, s)
          : launch(MatrixLogits<false>{logits, ld}, balance_bias, r, tokens, topk_idx, gates,
                   nullptr, align, s);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
