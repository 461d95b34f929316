// linear.hip — moe_linear and moe_linear_e4m3: one dense product with
// block-FP8 weights and E4M3 activations,
//   out[t][n] = sum_kb s[n/128][kb] * sum_{k in kb} a[t][k] * dec(w[n][k]) (+ bias[n]).
//
// bf16 output: the inner sum of one 128-column block is one matrix
// instruction (v_mfma_scale_f32_16x16x128_f8f6f4) over 16 weight rows and 16
// activation rows. The activations' power-of-two scale is the instruction's
// own E8M0 scale; the weights' fp32 block scale, which is no power of two,
// multiplies the instruction's fp32 result as it is added to the running sum.
// The instruction sums eight consecutive products of a lane on one grid, 2^-13
// of the largest (measured: 2^16 + 2^3 is exact, 2^16 + 2^2 loses the second
// term), so a sum errs by at most 2^-10 of its terms' magnitudes and, as the
// cuts go either way, by a few 2^-15 in norm: far below the output's own step
// of 2^-8.
//
// fp32 output: that error would be the result's, so the codes are widened to
// fp16 in registers (exact) and go through v_mfma_f32_16x16x32_f16, which
// keeps 2^-24 of the largest of eight products; the activations' scale is
// applied to the instruction's result.
//
// Weights are the instruction's A operand, so that a lane ends with four
// consecutive output features of one row.
#include "device.hpp"
#include "layer.hpp"

namespace moe {

constexpr int kLinB = 128;  // columns per scale block

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct LinearArgs {
  const uint8_t* codes;  // [M][K]
  const uint8_t* exps;   // [M][K/128]
  const uint8_t* w;      // [N][K]
  const float* ws;       // [ceil(N/128)][K/128]
  const float* bias;     // [N] or null
  void* out;
  int64_t M, ld_out;
  int N, K;
};

__device__ __forceinline__ i32x8_t operand(uint4 a, uint4 b) {
  i32x8_t v;
  v[0] = (int)a.x; v[1] = (int)a.y; v[2] = (int)a.z; v[3] = (int)a.w;
  v[4] = (int)b.x; v[5] = (int)b.y; v[6] = (int)b.z; v[7] = (int)b.w;
  return v;
}

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
__device__ __forceinline__ f16x8_t widen(int lo, int hi) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 v = {__builtin_bit_cast(uint32_t, e4m3x2_to_f16x2<false>(lo)),
                   __builtin_bit_cast(uint32_t, e4m3x2_to_f16x2<true>(lo)),
                   __builtin_bit_cast(uint32_t, e4m3x2_to_f16x2<false>(hi)),
                   __builtin_bit_cast(uint32_t, e4m3x2_to_f16x2<true>(hi))};
  return __builtin_bit_cast(f16x8_t, v);
}

// acc += s * 2^(scale - 127) * (A B over 128 k): lane l holds row l % 16 of
// each operand and the 32 k of its quarter l / 16 (any 32, the same for both
// operands); the result's column l % 16 (B's row) at rows 4 (l / 16) + v.
// scale: the E8M0 byte of B's row; s: the weights' block scale, premultiplied
// as block_scale() does.
// A sum of 128 code products reaches 2^25 and the activations' scale 2^120, so
// a factor is held back until s joins: the FP8 instruction's A operand has the
// constant scale 2^-kHold; the fp16 form takes what is above 2^100 out of 2^e.
constexpr int kHold = 18;
template <bool BF16>
__device__ __forceinline__ float block_scale(float s) {
  return BF16 ? s * (float)(1 << kHold) : s;
}
template <bool BF16>
__device__ __forceinline__ void mma128(f32x4& acc, const i32x8_t& a, const i32x8_t& b, int scale,
                                       float s) {
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
  if (BF16) {
    d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, d, 0, 0, 0, 127 - kHold, 0, scale);
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = fmaf(s, d[v], acc[v]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    d = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(a[2 * j], a[2 * j + 1]),
                                               widen(b[2 * j], b[2 * j + 1]), d, 0, 0, 0);
  const int e = scale - 127, e0 = e < 100 ? e : 100;
  const float se = __builtin_ldexpf(s, e - e0);
#pragma unroll
  for (int v = 0; v < 4; ++v) acc[v] = fmaf(se, __builtin_ldexpf(d[v], e0), acc[v]);
}

template <bool BF16>
__device__ __forceinline__ void store_out(void* out, int64_t at, float v) {
  if (BF16)
    reinterpret_cast<uint16_t*>(out)[at] = (uint16_t)f32_to_bf16_bits(v);
  else
    reinterpret_cast<float*>(out)[at] = v;
}

// One wavefront per tile of 16 output features x 16 rows, operands straight
// from global memory.
template <bool BF16>
__global__ __launch_bounds__(256) void linear_tile16(LinearArgs p) {
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int n0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * 16;
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  if (n0 >= p.N) return;
  const int nr = n0 + l16 < p.N ? n0 + l16 : p.N - 1;
  const int64_t mr = m0 + l16 < p.M ? m0 + l16 : p.M - 1;
  const int KB = p.K / kLinB;
  const uint8_t* wp = p.w + (size_t)nr * p.K + 16 * q;
  const uint8_t* ap = p.codes + (size_t)mr * p.K + 16 * q;
  const uint8_t* ep = p.exps + (size_t)mr * KB;
  const float* sp = p.ws + (size_t)(n0 / kLinB) * KB;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int kb = 0; kb < KB; ++kb) {
    const i32x8_t a = operand(ld16(wp + kb * kLinB), ld16(wp + kb * kLinB + 64));
    const i32x8_t b = operand(ld16(ap + kb * kLinB), ld16(ap + kb * kLinB + 64));
    mma128<BF16>(acc, a, b, ep[kb], block_scale<BF16>(sp[kb]));
  }
  if (m0 + l16 >= p.M) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int n = n0 + 4 * q + v;
    if (n < p.N) store_out<BF16>(p.out, mr * p.ld_out + n, acc[v] + (p.bias ? p.bias[n] : 0.f));
  }
}

static size_t al256(size_t n) { return (n + 255) / 256 * 256; }

static hipError_t launch_linear(const LinearArgs& p, bool bf16, hipStream_t s) {
  const dim3 grid((unsigned)((p.N + 63) / 64), (unsigned)((p.M + 15) / 16));
  if (bf16)
    linear_tile16<true><<<grid, 256, 0, s>>>(p);
  else
    linear_tile16<false><<<grid, 256, 0, s>>>(p);
  return hipGetLastError();
}

static moe_status check_sizes(int64_t M, int32_t N, int32_t K) {
  if (M < 0 || N <= 0 || K <= 0) return MOE_ERR_SHAPE;
  if (K % kLinB != 0) return MOE_ERR_UNSUPPORTED;
  // the tiles' row index, and the quantiser's grid
  if (M > (1 << 20) || M * (K / kLinB) >= ((int64_t)1 << 27)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

static moe_status linear_call(const void* x, int64_t ld_x, LinearArgs p, moe_dtype out_dtype,
                              void* workspace, size_t workspace_bytes, hipStream_t s) {
  const moe_status st = check_sizes(p.M, p.N, p.K);
  if (st != MOE_OK) return st;
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return MOE_ERR_SHAPE;
  if (p.ld_out < p.N || (x && ld_x < p.K)) return MOE_ERR_SHAPE;
  if (p.M == 0) return MOE_OK;
  const auto odd16 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 != 0; };
  if (odd16(x) || odd16(p.codes) || odd16(p.w) || (x && ld_x % 8 != 0)) return MOE_ERR_UNSUPPORTED;
  const size_t need = moe_linear_workspace_bytes(p.M, p.N, p.K, x ? 0 : 1);
  if (need > 0) {
    if (!workspace) return MOE_ERR_NULL;
    if (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
      return MOE_ERR_WORKSPACE;
  }
  if (x) {
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    uint8_t* exps = codes + al256((size_t)p.M * p.K);
    if (launch_quant_act(x, p.M, p.K, codes, exps, s, ld_x) != hipSuccess) return MOE_ERR_HIP;
    p.codes = codes;
    p.exps = exps;
  }
  return launch_linear(p, out_dtype == MOE_BF16, s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_linear_workspace_bytes(int64_t rows, int32_t out_features, int32_t in_features,
                                  int32_t x_is_codes) {
  if (check_sizes(rows, out_features, in_features) != MOE_OK || rows == 0) return 0;
  return x_is_codes ? 0
                    : al256((size_t)rows * in_features) +
                          al256((size_t)rows * (in_features / kLinB));
}

moe_status moe_linear(const void* x, int64_t ld_x, const uint8_t* w, const float* w_scales,
                      const float* bias, int64_t rows, int32_t out_features, int32_t in_features,
                      void* out, int64_t ld_out, moe_dtype out_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!x || !w || !w_scales || !out) return MOE_ERR_NULL;
  const LinearArgs p{nullptr, nullptr, w,    w_scales,     bias,
                     out,     rows,    ld_out, out_features, in_features};
  return linear_call(x, ld_x, p, out_dtype, workspace, workspace_bytes,
                     static_cast<hipStream_t>(stream));
}

moe_status moe_linear_e4m3(const uint8_t* codes, const uint8_t* exps, const uint8_t* w,
                           const float* w_scales, const float* bias, int64_t rows,
                           int32_t out_features, int32_t in_features, void* out, int64_t ld_out,
                           moe_dtype out_dtype, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (!codes || !exps || !w || !w_scales || !out) return MOE_ERR_NULL;
  const LinearArgs p{codes, exps, w, w_scales, bias, out, rows, ld_out, out_features, in_features};
  return linear_call(nullptr, 0, p, out_dtype, workspace, workspace_bytes,
                     static_cast<hipStream_t>(stream));
}

}  // extern "C"
