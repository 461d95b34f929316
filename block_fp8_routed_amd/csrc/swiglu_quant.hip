// swiglu_quant.hip — moe_swiglu_quantize_e4m3: h = silu(gate) * up of a
// [gate | up] matrix, written as E4M3 bytes with one power-of-two scale per
// row and 128 columns: what stands between the two products of a dense
// block-FP8 feed-forward block (moe_linear, then moe_linear_e4m3).
//
// h is computed in fp32 and quantised by the activation quantiser's rule
// (e4m3_round.hpp). An h that is NaN (only from a NaN or infinite input)
// becomes the NaN byte and does not take part in its block's scale; one
// beyond fp32 counts as the largest finite value.
//
// Bound by memory (4 bytes read and 1 + 1/128 written per element) as long as
// an element takes no more than some 20 instructions: the exponential and the
// quotient are written out below, and the row of a chunk is found by a
// multiplication. Sixteen lanes per block (a DPP row), eight columns of the
// gate and of the up half per lane with one 16-byte load each. Measured: 8191 x
// 4096 outputs 27.7 us (168 MB, 6.1 TB/s; 179 instructions a wavefront of 512
// outputs), 4 x 1024 2.0 us (a launch).
#include <float.h>

#include "device.hpp"
#include "e4m3_round.hpp"
#include "layer.hpp"

namespace moe {

// silu(g) * u. e^-g = 2^t 2^r with t = -g log2(e) rounded to fp32 and r the
// rest of the product (an fma against the same constant, plus the constant's
// own rest), 2^r = 1 + r ln 2 (r grows with t's step: what is left out is 2^-42 at
// |g| = 20 and 2^-38 at 69); the quotient is the hardware reciprocal with one
// Newton step. About 2 ulps in all.
__device__ __forceinline__ float swiglu1(float g, float u) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float t = -g * kLog2e;
  const float r = fmaf(-g, kLog2e, -t) - g * kLog2eRest;
  const float p = __builtin_amdgcn_exp2f(t);
  const float d = 1.0f + fmaf(p, r * kLn2, p);
  float q = __builtin_amdgcn_rcpf(d);
  q = fmaf(q, fmaf(-d, q, 1.0f), q);
  return g * q * u;
}

// thread i of the grid takes columns 8 (i % 16) .. + 7 of block i / 16
__global__ __launch_bounds__(256) void swiglu_quant_kernel(const uint16_t* __restrict__ gu,
                                                          int64_t ld, uint32_t n, int I,
                                                          FastDiv by_row,
                                                          uint2* __restrict__ codes,
                                                          uint8_t* __restrict__ exps) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x, c = i < n ? i : n - 1;
  const uint32_t row = by_row.div(c), col = 8 * (c - row * (uint32_t)(I / 8));
  const uint16_t* src = gu + row * ld + col;
  const uint4 gw = ld16_nt(src), uw = ld16_nt(src + I);
  const uint32_t gd[4] = {gw.x, gw.y, gw.z, gw.w}, ud[4] = {uw.x, uw.y, uw.z, uw.w};
  float g[8], u[8], h[8];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    g[j] = j & 1 ? bf16_hi(gd[j / 2]) : bf16_lo(gd[j / 2]);
    u[j] = j & 1 ? bf16_hi(ud[j / 2]) : bf16_lo(ud[j / 2]);
    h[j] = swiglu1(g[j], u[j]);
    m = max(m, __float_as_uint(h[j]) & 0x7fffffffu);
  }
  // Gates down from -69 (e^69 = 2^99.5), where the reciprocal nears its end, and
  // infinite or NaN values are computed again in full (an infinite h counts as the
  // largest finite value). Each value goes by its own gate and result, so that
  // neighbours in the wavefront, which may be other rows, have no say in it.
  uint2 nans = make_uint2(0u, 0u);  // 0x7f at the bytes whose h is NaN
  if (__ballot(m >= 0x7f800000u || bf16x8_max_bits(gw) >= 0xc28au)) {
    m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = h[j];
      if (g[j] <= -69.0f || !(fabsf(v) <= FLT_MAX)) {
        v = g[j] / (1.0f + expf(-g[j])) * u[j];
        if (fabsf(v) > FLT_MAX) v = copysignf(FLT_MAX, v);
      }
      const uint32_t bits = __float_as_uint(v), mag = bits & 0x7fffffffu;
      const bool nan = mag > 0x7f800000u;
      h[j] = nan ? 0.f : v;
      (j < 4 ? nans.x : nans.y) |= nan ? 0x7fu << (8 * (j & 3)) : 0u;
      m = max(m, nan ? 0u : mag);
    }
  }
  const int e = act_exponent(__uint_as_float(row16_max_u32(m)));
  if (i >= n) return;
  uint2 q = e4m3x8_of_f32(h, e);
  q.x |= nans.x;  // (their h was replaced by 0)
  q.y |= nans.y;
  codes[i] = q;
  if ((i & 15) == 0) exps[i >> 4] = (uint8_t)(e + 127);
}

}  // namespace moe

extern "C" moe_status moe_swiglu_quantize_e4m3(const void* gate_up, int64_t ld, int64_t tokens,
                                               int32_t inter, uint8_t* codes, uint8_t* exps,
                                               void* stream) {
  using namespace moe;
  if (!gate_up || !codes || !exps) return MOE_ERR_NULL;
  if (tokens < 0 || inter <= 0 || ld < 2 * (int64_t)inter) return MOE_ERR_SHAPE;
  if (inter % kActBlock != 0 || ld % 8 != 0 || reinterpret_cast<uintptr_t>(gate_up) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(codes) % 8 != 0)
    return MOE_ERR_UNSUPPORTED;
  const int64_t nb = tokens * (inter / kActBlock);
  if (nb >= ((int64_t)1 << 27)) return MOE_ERR_UNSUPPORTED;  // the grid's x dimension
  if (tokens == 0) return MOE_OK;
  const uint32_t n = (uint32_t)(nb * (kActBlock / 8));
  swiglu_quant_kernel<<<(n + 255) / 256, 256, 0, static_cast<hipStream_t>(stream)>>>(
      static_cast<const uint16_t*>(gate_up), ld, n, inter, FastDiv::of((uint32_t)inter / 8),
      reinterpret_cast<uint2*>(codes), exps);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
