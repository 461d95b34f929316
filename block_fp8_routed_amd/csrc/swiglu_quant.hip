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
// Bound by memory: 4 bytes read and 1 + 1/128 written per element. Sixteen
// lanes per block (a DPP row), eight columns of the gate and of the up half
// per lane with one 16-byte load each.
#include <float.h>

#include "device.hpp"
#include "e4m3_round.hpp"
#include "layer.hpp"

namespace moe {

// thread i of the grid takes columns 8 (i % 16) .. + 7 of block i / 16
__global__ __launch_bounds__(256) void swiglu_quant_kernel(const uint16_t* __restrict__ gu,
                                                          int64_t ld, int64_t nblocks, int I,
                                                          uint2* __restrict__ codes,
                                                          uint8_t* __restrict__ exps) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t n = nblocks * (kActBlock / 8);
  const int64_t c = i < n ? i : n - 1;
  const int per_row = I / 8;
  const int64_t row = c / per_row;
  const int col = (int)(c - row * per_row) * 8;
  const uint16_t* src = gu + row * ld + col;
  const uint4 gw = ld16(src), uw = ld16(src + I);
  const uint32_t gd[4] = {gw.x, gw.y, gw.z, gw.w}, ud[4] = {uw.x, uw.y, uw.z, uw.w};
  float h[8];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float g = j & 1 ? bf16_hi(gd[j / 2]) : bf16_lo(gd[j / 2]);
    const float u = j & 1 ? bf16_hi(ud[j / 2]) : bf16_lo(ud[j / 2]);
    float v = g / (1.0f + expf(-g)) * u;
    if (fabsf(v) > FLT_MAX) v = copysignf(FLT_MAX, v);
    h[j] = v;
    m = max(m, v == v ? __float_as_uint(fabsf(v)) : 0u);
  }
  const int e = act_exponent(__uint_as_float(row16_max_u32(m)));
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    q[j] = h[j] == h[j] ? e4m3_rne(__builtin_ldexpf(h[j], -e)) : 0x7fu;
  if (i >= n) return;
  codes[i] = make_uint2(q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24),
                        q[4] | (q[5] << 8) | (q[6] << 16) | (q[7] << 24));
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
  const int64_t chunks = nb * (kActBlock / 8);
  swiglu_quant_kernel<<<(unsigned)((chunks + 255) / 256), 256, 0,
                        static_cast<hipStream_t>(stream)>>>(
      static_cast<const uint16_t*>(gate_up), ld, nb, inter, reinterpret_cast<uint2*>(codes),
      exps);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}
