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
// computes just the drawn experts' scores (or the groups') in fp64. The gates
// are fp64 rounded once.
//
// A masked expert (logit NaN or not above -3.3e38, which takes -inf and the
// lowest finite value of fp32 and bf16) has score 0, adds nothing to its
// group and is chosen only when the kept groups run out of others (then the
// lowest index first, gate 0).
//
// One wavefront per token. Lane L owns nv consecutive experts L nv, L nv + 1,
// ...: the lowest lane that holds a value then holds the lowest expert with
// it, and where nv divides the group size a lane lies in one group.
#include <cmath>

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

// e^x in fp64 for x up to 709, within 2^-49: x = n ln 2 + r, |r| <= 0.35,
// and the exponential series to r^12 (the rest is below 2^-50).
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

// LDS of one wavefront. Expert i of lane L is at L NV + i.
template <int NV>
struct GateLds {
  float raw[64 * NV];     // logits, -inf for masked and absent experts
  uint64_t key[64 * NV];  // choose_exact: order keys of c
  union {
    uint32_t head[2][64];  // each lane's two largest keys; the ranked choice
    double pair[2][64];    // exact_groups: each lane's two largest c
  };
};

// The wavefront's own LDS traffic is in order; this keeps the compiler to it.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// The softmax's sum of e^(l - top) over the lane's NV logits and the wavefront.
template <int NV>
__device__ __forceinline__ double softmax_sum(const float* raw, float top) {
  double z = 0.0;
#pragma unroll 2
  for (int i = 0; i < NV; ++i) z += exp64((double)raw[i] - (double)top);  // (-inf adds 0)
  return wave_sum_f64(z);
}

// An expert's score from its logit (-inf: masked); softmax: not yet divided
// by the sum.
__device__ __forceinline__ double score64(const GateRule& r, float logit, float top) {
  const double x = r.softmax ? (double)logit - (double)top : fmin(-(double)logit, 709.0);
  const double e = exp64(x);
  const double s = r.softmax ? e : 1.0 / (1.0 + e);
  return logit > kMaskedLogit ? s : 0.0;
}

// The groups that come first by their scores in lanes 0 .. groups - 1 (keys),
// as a mask.
__device__ __forceinline__ unsigned long long first_groups(const GateRule& r, uint64_t key) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int j = 0; j < r.groups; ++j) {
    const uint64_t o = readlane_u64(key, j);
    before += o > key || (o == key && j < lane) ? 1 : 0;
  }
  return __ballot(lane < r.groups && before < r.top_groups);
}

// The choice by fp64 keys, for any group size: lane j < top_k gets the j-th
// (as a slot of GateLds). Rolled loops over LDS: it runs for few tokens.
template <int NV>
__device__ __forceinline__ int choose_exact(const GateRule& r, float top,
                                            const float* __restrict__ balance, GateLds<NV>& lds) {
  const int lane = threadIdx.x & 63, e0 = lane * r.nv;
  const float* raw = lds.raw + lane * NV;
  uint64_t* key = lds.key + lane * NV;
  const double z = r.softmax ? softmax_sum<NV>(raw, top) : 1.0;
#pragma unroll 1
  for (int i = 0; i < r.nv; ++i) {
    const int e = e0 + i;
    const float v = raw[i];
    double c = score64(r, v, top);
    if (r.softmax) c = z > 0.0 ? c / z : 0.0;
    if (balance && e < r.experts) c += (double)balance[e];
    key[i] = e < r.experts ? (v > kMaskedLogit ? order_key(c) : kKeyMasked) : kKeyAbsent;
  }
  wave_lds_fence();
  if (r.groups > 1) {
    double gs = -INFINITY;  // lane g: group g's score
    for (int g = 0; g < r.groups; ++g) {
      // the group's two largest keys, lanes taking every 64th expert
      uint64_t a = 0, b = 0;
      for (int j = lane; j < r.per_group; j += 64) {
        const int e = g * r.per_group + j, l = e / r.nv;
        const uint64_t c = lds.key[l * NV + e - l * r.nv];
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
      double s = m > kKeyMasked ? key_value(m) : -INFINITY;
      if (r.rank > 1 && m2 > kKeyMasked) s += key_value(m2);
      if (lane == g) gs = s;
    }
    const unsigned long long kept = first_groups(r, gs > -INFINITY ? order_key(gs) : kKeyMasked);
#pragma unroll 1
    for (int i = 0; i < r.nv; ++i)
      if (e0 + i < r.experts && !((kept >> ((e0 + i) / r.per_group)) & 1)) key[i] = kKeyAbsent;
  }
  uint64_t best = 0;  // the lane's largest key and its lowest place
  int place = 0;
  const auto rescan = [&] {
    best = 0;
#pragma unroll 1
    for (int i = 0; i < r.nv; ++i)
      if (key[i] > best) {
        best = key[i];
        place = i;
      }
  };
  rescan();
  int mine = 0;
  for (int j = 0; j < r.top_k; ++j) {
    const uint64_t m = wave_max_u64(best);
    const int wl = __ffsll((unsigned long long)__ballot(best == m)) - 1;
    const int slot = wl * NV + __builtin_amdgcn_readlane(place, wl);
    if (lane == j) mine = slot;
    if (lane == wl) {
      key[place] = kKeyAbsent;
      rescan();
    }
  }
  return mine;
}

// The kept groups by fp64 scores, as a mask of groups, where every lane lies
// in one group.
template <int NV>
__device__ __forceinline__ unsigned long long exact_groups(const GateRule& r, float top,
                                                           const float* __restrict__ balance,
                                                           GateLds<NV>& lds) {
  const int lane = threadIdx.x & 63, e0 = lane * r.nv;
  const float* raw = lds.raw + lane * NV;
  const double z = r.softmax ? softmax_sum<NV>(raw, top) : 1.0;
  double a = -INFINITY, b = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < r.nv; ++i) {
    double c = score64(r, raw[i], top) / z;
    if (balance && e0 + i < r.experts) c += (double)balance[e0 + i];
    if (!(raw[i] > kMaskedLogit)) c = -INFINITY;
    b = fmax(b, fmin(a, c));
    a = fmax(a, c);
  }
  wave_lds_fence();
  lds.pair[0][lane] = a;
  lds.pair[1][lane] = b;
  wave_lds_fence();
  a = b = -INFINITY;
  if (lane < r.groups)
    for (int j = 0; j < r.group_lanes; ++j) {
      const double c = lds.pair[0][lane * r.group_lanes + j];
      b = fmax(fmax(b, fmin(a, c)), lds.pair[1][lane * r.group_lanes + j]);
      a = fmax(a, c);
    }
  const double gs = r.rank > 1 && b > -INFINITY ? a + b : a;
  wave_lds_fence();
  return first_groups(r, a > -INFINITY ? order_key(gs) : kKeyMasked);
}

__device__ __forceinline__ bool uniform_bool(bool b) { return __ballot(b) != 0ull; }

// A uniform value that the compiler takes for one per lane.
__device__ __forceinline__ float uniform(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

// fp32 values as unsigned keys in the same order (no NaN).
__device__ __forceinline__ uint32_t order32(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value32(uint32_t h) {
  return __uint_as_float(h ^ ((uint32_t)((int32_t)~h >> 31) | 0x80000000u));
}

// The choice by fp32 keys, made exact where they are close. False: not
// possible this way (masked experts have to be chosen, or more than
// kCandidates are too close to tell). Lane j < top_k gets the j-th expert (as
// a slot of GateLds).
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
//   The wavefront draws the largest key top_k times, and on while the next one
// is close to the last of these. If any two neighbours are close, the drawn
// ones (one per lane) are ranked by fp64 c and index.
constexpr int kCandidates = 32;
template <int NV, bool BF16>
__device__ __forceinline__ bool choose_fast(const GateRule& r, const float (&v)[NV], float top,
                                            const float (&bias)[NV],
                                            const float* __restrict__ balance, GateLds<NV>& lds,
                                            int& mine) {
  constexpr int kLow = NV <= 1 ? 0 : NV <= 2 ? 1 : NV <= 4 ? 2 : NV <= 8 ? 3 : 4;
  constexpr uint32_t kPlace = (1u << kLow) - 1u;
  const int lane = threadIdx.x & 63;
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
    z = uniform(group_sum<64>(z));
    const float q = z > 0.f ? 1.0f / z : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = fmaf(c[i], q, bias[i]);
    eps = uniform(0x1p-18f * q + 0x1p-22f);
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
    lds.head[0][lane] = key[0] >> kLow;
    if constexpr (NV > 1) lds.head[1][lane] = key[1] >> kLow;
    wave_lds_fence();
    const int lg = r.group_lanes;
    uint32_t a = 0, b = 0;
    for (int j0 = 0; j0 < lg; j0 += 8) {  // eight lanes' keys requested together
      uint32_t x[8], y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = lane * lg + j0 + j;
        x[j] = lds.head[0][at < 64 ? at : 63];
        if constexpr (NV > 1) y[j] = lds.head[1][at < 64 ? at : 63];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j0 + j >= lg) x[j] = 0;
        b = max(b, min(a, x[j]));
        a = max(a, x[j]);
        if constexpr (NV > 1) b = max(b, j0 + j < lg ? y[j] : 0u);
      }
    }
    const bool in = lane < r.groups, two = r.rank > 1 && b != 0u;
    const float av = value32(a << kLow), bv = two ? value32(b << kLow) : 0.f;
    const float gs = in && a != 0u ? av + bv : -INFINITY;
    const float mag = a != 0u ? fabsf(av) + fabsf(bv) : 0.f;
    int before = 0;
    for (int j = 0; j < r.groups; ++j) {
      const float o = readlane_f(gs, j);
      before += o > gs || (o == gs && j < lane) ? 1 : 0;
    }
    unsigned long long kept = __ballot(in && before < r.top_groups);
    if (r.top_groups < r.groups) {
      // the last group kept and the first one dropped
      const int lk = __ffsll(__ballot(in && before == r.top_groups - 1)) - 1;
      const int ld = __ffsll(__ballot(in && before == r.top_groups)) - 1;
      const float sk = readlane_f(gs, lk), sd = readlane_f(gs, ld);
      const float m = fmaxf(readlane_f(mag, lk), readlane_f(mag, ld));
      // (a bf16 logit loses nothing to its place's bits: equal keys are equal scores)
      const bool sure = by_logit ? sk > -INFINITY && (!close(sk, sd) || (BF16 && sk == sd))
                                 : sk - sd > 4.0f * eps + 4.0f * kCut * m;
      if (!sure) kept = exact_groups(r, top, balance, lds);
    }
    const int own = (int)(((float)lane + 0.5f) * r.inv_group_lanes);
    const bool mykept = own < r.groups && ((kept >> own) & 1);
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = mykept ? key[i] : 0u;
  }
  uint32_t got = 0, m = 0;  // lane j: the j-th key; the last one drawn
  mine = 0;
  // draws the largest key m (found before) as the n-th
  const auto draw = [&](uint32_t h, int n) {
    const int wl = __ffsll((unsigned long long)__ballot(h == m)) - 1;
    const int wi = (int)(kPlace - ((uint32_t)__builtin_amdgcn_readlane((int)key[0], wl) & kPlace));
    got = lane == n ? m : got;
    mine = lane == n ? wl * NV + wi : mine;
    const bool pop = lane == wl;
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = pop ? (i + 1 < NV ? key[i + 1] : 0u) : key[i];
  };
  for (int j = 0; j < r.top_k; ++j) {
    const uint32_t h = key[0] >> kLow;
    m = wave_max_u32(h);
    draw(h, j);
  }
  if (m == 0u) return false;
  const float last = value32(m << kLow);
  int n = r.top_k;
  for (;; ++n) {
    const uint32_t h = key[0] >> kLow;
    m = wave_max_u32(h);
    if (m == 0u || !uniform_bool(close(last, value32(m << kLow)))) break;
    if (n == kCandidates) return false;
    draw(h, n);
  }
  // neighbours: far enough apart, or the same numbers (the lower index came first)
  const float x = value32(got << kLow), y = __shfl_down(x, 1);
  const float lj = lds.raw[mine], ln = __shfl_down(lj, 1);
  const bool unsure = lane + 1 < n && close(x, y) && (balance || lj != ln);
  if (n > r.top_k || __ballot(unsure)) {
    const int l = mine / NV, e = l * r.nv + mine - l * NV;
    double cx = score64(r, lj, top);
    if (balance) {
      if (r.softmax) cx /= softmax_sum<NV>(lds.raw + lane * NV, top);
      cx += (double)balance[e];
    }
    const uint64_t ck = order_key(cx);
    int before = 0;
    for (int j = 0; j < n; ++j) {
      const uint64_t o = readlane_u64(ck, j);
      const int oe = __builtin_amdgcn_readlane(e, j);
      before += o > ck || (o == ck && oe < e) ? 1 : 0;
    }
    wave_lds_fence();
    if (lane < n) lds.head[0][before] = (uint32_t)mine;
    wave_lds_fence();
    mine = lane < r.top_k ? (int)lds.head[0][lane] : 0;
  }
  return true;
}

template <int NV, class Logits, bool BALANCE>
__global__ __launch_bounds__(256) void gate_select_kernel(Logits lg,
                                                         const float* __restrict__ balance_,
                                                         GateRule r, int64_t T,
                                                         int32_t* __restrict__ topk,
                                                         float* __restrict__ gates,
                                                         int32_t* __restrict__ zero_word) {
  __shared__ GateLds<NV> all[4];
  if (zero_word && blockIdx.x == 0 && threadIdx.x == 0) *zero_word = 0;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= T) return;  // (no workgroup barrier follows)
  GateLds<NV>& lds = all[wave];
  const float* balance = BALANCE ? balance_ : nullptr;
  const int e0 = lane * r.nv;
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
    lds.raw[lane * NV + i] = v[i];
  }
  // (a token without any expert left: 0, so that no difference is NaN)
  if (r.softmax) top = fmaxf(wave_max_f32(top), -3.402823466e38f);
  top = uniform(top);
  wave_lds_fence();
  int mine = 0;
  if (!(r.fast && choose_fast<NV, Logits::kBf16>(r, v, top, bias, balance, lds, mine)))
    mine = choose_exact<NV>(r, top, balance, lds);
  // gates
  double s = lane < r.top_k ? score64(r, lds.raw[mine], top) : 0.0;
  double den = 1.0;
  if (r.renorm) {
    den = s;
#pragma unroll
    for (int o = 8; o; o >>= 1) den += __shfl_xor(den, o, 16);
  } else if (r.softmax) {
    den = softmax_sum<NV>(lds.raw + lane * NV, top);
  }
  if (lane < r.top_k) {
    const int l = mine / NV;
    topk[t * r.top_k + lane] = l * r.nv + mine - l * NV;
    gates[t * r.top_k + lane] = (float)(den > 0.0 ? s / den * (double)r.scale : 0.0);
  }
}

template <class Logits>
static hipError_t launch(const Logits& lg, const float* balance, GateRule r, int64_t T,
                         int32_t* topk, float* gates, int32_t* zero_word, bool vec, hipStream_t s) {
  const dim3 grid((unsigned)((T + 3) / 4));
  const int nv = r.nv;
  const int full = nv <= 1 ? 1 : nv <= 2 ? 2 : nv <= 4 ? 4 : nv <= 8 ? 8 : 16;
  r.vec = vec && nv == full && r.experts % nv == 0;
#define MOE_GATE(NV)                                                                          \
  balance ? gate_select_kernel<NV, Logits, true><<<grid, 256, 0, s>>>(lg, balance, r, T, topk, \
                                                                      gates, zero_word)       \
          : gate_select_kernel<NV, Logits, false><<<grid, 256, 0, s>>>(lg, nullptr, r, T, topk, \
                                                                       gates, zero_word)
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
  // experts per lane: the fewest that cover all; with groups, of those that
  // divide a group, if there is one up to 16
  const int least = (experts + 63) / 64;
  r->nv = least;
  r->fast = true;
  if (g->groups > 1) {
    while (r->nv <= 16 && per % r->nv != 0) ++r->nv;
    r->fast = r->nv <= 16;
    if (!r->fast) r->nv = least;
  }
  r->group_lanes = r->fast ? per / r->nv : 0;
  r->inv_group_lanes = r->fast ? 1.0f / (float)r->group_lanes : 0.f;
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
                topk, gates, zero_word, false, s);
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
  // vector loads of a lane's experts: rows and the first of each lane 16-byte
  // aligned, or as far as a lane's experts reach
  const int64_t size = dtype == MOE_BF16 ? 2 : 4, span = r.nv * size < 16 ? r.nv * size : 16;
  const bool vec = reinterpret_cast<uintptr_t>(logits) % span == 0 && ld * size % span == 0;
  const hipError_t e =
      dtype == MOE_BF16
          ? launch(MatrixLogits<true>{logits, ld}, balance_bias, r, tokens, topk_idx, gates,
                   nullptr, vec, s)
          : launch(MatrixLogits<false>{logits, ld}, balance_bias, r, tokens, topk_idx, gates,
                   nullptr, vec, s);
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
