// quant_act.hip — moe_quantize_act_e4m3: bf16 activations to E4M3 bytes with
// one power-of-two scale per token and block of 128 columns.
//
// This is the activation side of the variant that runs both operands of both
// expert contractions in E4M3 at prefill sizes. The pages describe E4M3
// weights only (colizig page, "What this project is trying to prove":
// natively block-FP8 checkpoints); the activation side is a reading of this
// project: a block's scale is 2^e with e the smallest integer such that the
// block's largest magnitude is at most 448 * 2^e (0 for an all-zero block,
// never below -127), and each value becomes the nearest E4M3FN value of
// x * 2^-e, an exact tie going to the even mantissa, the sign kept (negative
// values that round to zero give -0). Power-of-two scales are what gfx950's
// block-scaled FP8 matrix instructions take (E8M0), so the scale can ride in
// the instruction itself.
//
// The conversion instruction takes 2^e itself and rounds x * 2^-e once, so
// each code is decided exactly as an exact-arithmetic rounding would.
//
// Sixteen lanes per block (a DPP row): lane L of a row takes columns 8L ..
// 8L + 7 with one 16-byte load, and the block's largest magnitude comes from
// a four-step DPP maximum within the row over the lanes' bf16 bit patterns
// (non-negative floats order as unsigned integers). Bound by memory: 8192 x
// 4096 19 us (101 MB, 5.3 TB/s).
#include "device.hpp"
#include "e4m3_round.hpp"
#include "layer.hpp"

namespace moe {

// thread i of the grid takes 16-byte chunk i (columns 8 (i % 16) .. + 7 of
// block i / 16); chunks past the end repeat the last one and store nothing.
// STRIDED: rows of per_row chunks, ld_chunks apart (else one after the other).
// x is read and the codes written once each, non-temporally.
template <bool STRIDED>
__global__ __launch_bounds__(256) void quant_act_kernel(const uint4* __restrict__ x, uint32_t n,
                                                       uint2* __restrict__ codes,
                                                       uint8_t* __restrict__ exps, int per_row,
                                                       FastDiv by_row, int64_t ld_chunks) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x, c = i < n ? i : n - 1;
  int64_t src = c;
  if (STRIDED) {
    const uint32_t row = by_row.div(c);
    src = row * ld_chunks + (c - row * (uint32_t)per_row);
  }
  const uint4 w = ld16_nt(x + src);
  const int e = act_exponent(__uint_as_float(row16_max_u32(bf16x8_max_abs(w)) << 16));
  if (i >= n) return;
  const uint2 q = e4m3x8_of_bf16(w, e);
  codes[i] = q;
  if ((i & 15) == 0) exps[i >> 4] = (uint8_t)(e + 127);
}

hipError_t launch_quant_act(const void* x, int64_t T, int H, uint8_t* codes, uint8_t* exps,
                            hipStream_t s, int64_t ld) {
  const uint32_t n = (uint32_t)(T * (H / 8));  // below 2^31 (the callers' limit on blocks)
  const unsigned grid = (n + 255) / 256;
  const uint4* src = static_cast<const uint4*>(x);
  uint2* dst = reinterpret_cast<uint2*>(codes);
  const FastDiv by_row = FastDiv::of((uint32_t)(H / 8));
  if (ld == 0 || ld == H)
    quant_act_kernel<false><<<grid, 256, 0, s>>>(src, n, dst, exps, H / 8, by_row, H / 8);
  else
    quant_act_kernel<true><<<grid, 256, 0, s>>>(src, n, dst, exps, H / 8, by_row, ld / 8);
  return hipGetLastError();
}

}  // namespace moe

extern "C" moe_status moe_quantize_act_e4m3(const void* x, int64_t tokens, int32_t hidden,
                                            uint8_t* codes, uint8_t* exps, void* stream) {
  if (!x || !codes || !exps) return MOE_ERR_NULL;
  if (tokens < 0 || hidden <= 0) return MOE_ERR_SHAPE;
  if (hidden % moe::kActBlock != 0) return MOE_ERR_UNSUPPORTED;
  if (tokens * (int64_t)(hidden / moe::kActBlock) >= ((int64_t)1 << 27))
    return MOE_ERR_UNSUPPORTED;  // the grid's x dimension counts 16-byte chunks / 256
  if (tokens == 0) return MOE_OK;
  return moe::launch_quant_act(x, tokens, hidden, codes, exps, static_cast<hipStream_t>(stream)) ==
                 hipSuccess
             ? MOE_OK
             : MOE_ERR_HIP;
}
