// linear_w4.hip — moe_linear_w4 and moe_grouped_linear_w4: the entry points, and the
// rows of x that the tiles take.
#include "linear_w4.hpp"

namespace moe {

// Columns 8 c .. 8 c + 7 in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 half_order(const uint4 v, int e) {
  const float f[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                      bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2_t h = {(_Float16)__builtin_ldexpf(f[i], -e), (_Float16)__builtin_ldexpf(f[i + 4], -e)};
    o[i] = __builtin_bit_cast(uint32_t, h);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The largest bf16 magnitude of eight, as its bits.
__device__ __forceinline__ uint32_t max_abs8(const uint4 v) {
  const auto two = [](uint32_t a) { return max((a & 0x7fffu), (a >> 16) & 0x7fffu); };
  return max(max(two(v.x), two(v.y)), max(two(v.z), two(v.w)));
}

// Rows of x as fp16 x 2^-e [M][Kp], zeros behind K, and e [M]. W wavefronts a row
// (1: four rows a workgroup). Rows of up to 512 kHold W columns are read once. Bound by
// its bytes: 32768 rows of 2048, 268 MB, 41 us (6.5 TB/s).
template <int W>
__global__ __launch_bounds__(256) void w4_halves(const uint16_t* __restrict__ x, int64_t ld_x,
                                                 int64_t M, int K, int Kp,
                                                 uint4* __restrict__ xh, int32_t* __restrict__ xe) {
  constexpr int kHold = 4;
  __shared__ uint32_t part[4];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + w : (int64_t)blockIdx.x;
  if (row >= M) return;
  const int first = W == 1 ? lane : (int)threadIdx.x, step = 64 * W;
  const uint4* src = reinterpret_cast<const uint4*>(x + row * ld_x);
  uint4 held[kHold];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int c = first + i * step;
    held[i] = 8 * c < K ? ld16(src + c) : make_uint4(0, 0, 0, 0);
    m = max(m, max_abs8(held[i]));
  }
  for (int c = first + kHold * step; 8 * c < K; c += step) m = max(m, max_abs8(ld16(src + c)));
  m = wave_max_u32(m);
  if (W > 1) {
    if (lane == 0) part[w] = m;
    __syncthreads();
    m = max(max(part[0], part[1]), max(part[2], part[3]));
  }
  // m = 2^(p - 127) times [1, 2) (a NaN or infinity counts as the largest binade)
  const int p = (int)(m >> 7) < 254 ? (int)(m >> 7) : 254;
  const int e = m == 0 ? 0 : p - 127 - 14;
  uint4* dst = xh + row * (Kp / 8);
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int c = first + i * step;
    if (8 * c < Kp) dst[c] = half_order(held[i], e);
  }
  for (int c = first + kHold * step; 8 * c < Kp; c += step)
    dst[c] = half_order(8 * c < K ? ld16(src + c) : make_uint4(0, 0, 0, 0), e);
  if (first == 0) xe[row] = e;
}

void launch_w4_halves(const W4Args& p, int Kp, uint4* xh, int32_t* xe, hipStream_t s) {
  if (p.K <= 2048)
    w4_halves<1><<<(unsigned)((p.M + 3) / 4), 256, 0, s>>>(p.x, p.ld_x, p.M, p.K, Kp, xh, xe);
  else
    w4_halves<4><<<(unsigned)p.M, 256, 0, s>>>(p.x, p.ld_x, p.M, p.K, Kp, xh, xe);
}

void launch_w4_group32(const W4Args& p, void* workspace, hipStream_t s);
void launch_w4_group64(const W4Args& p, void* workspace, hipStream_t s);
void launch_w4_group128(const W4Args& p, void* workspace, hipStream_t s);

static size_t w4_workspace(int64_t M, int E, int N, int K, bool bf16) {
  if (M == 0 || w4_form(M, E, N, K, bf16) != kW4Tiles) return 0;
  return w4_al256((size_t)M * w4_padded(K) * 2) + w4_al256((size_t)M * 4);
}

constexpr int kW4Limit = 1 << 20;  // rows, features, columns
static moe_status w4_call(W4Args p, int group, moe_dtype scale_dtype, moe_dtype out_dtype,
                          void* workspace, size_t workspace_bytes, hipStream_t s) {
  if (p.M < 0 || p.N <= 0 || p.K <= 0 || p.E <= 0 || group <= 0) return MOE_ERR_SHAPE;
  if (p.K % group != 0 || (p.swiglu && p.N % 2 != 0)) return MOE_ERR_SHAPE;
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return MOE_ERR_SHAPE;
  if (scale_dtype != MOE_F32 && scale_dtype != MOE_BF16) return MOE_ERR_SHAPE;
  if (p.ld_x < p.K || p.ld_out < (p.swiglu ? p.N / 2 : p.N)) return MOE_ERR_SHAPE;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
  if (p.E > kMaxExperts || p.K > kW4Limit || p.N > kW4Limit || p.M > kW4Limit)
    return MOE_ERR_UNSUPPORTED;
  // fewer than 2^32 threads a grid: 256 a tile of 32 rows and 128 features
  if (row_tiles(p, 32) * ((p.N + 127) / 128) >= ((int64_t)1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (p.M == 0) return MOE_OK;
  const auto odd = [](const void* q, int n) { return reinterpret_cast<uintptr_t>(q) % n != 0; };
  if (odd(p.x, 16) || odd(p.w, 16) || p.ld_x % 8 != 0 || odd(p.ws, scale_dtype == MOE_BF16 ? 2 : 4) ||
      odd(p.bias, 4) || odd(p.offsets, 4) || odd(p.out, out_dtype == MOE_BF16 ? 2 : 4))
    return MOE_ERR_UNSUPPORTED;
  const size_t need = w4_workspace(p.M, p.E, p.N, p.K, out_dtype == MOE_BF16);
  if (need > 0) {
    if (!workspace) return MOE_ERR_NULL;
    if (workspace_bytes < need || odd(workspace, 256)) return MOE_ERR_WORKSPACE;
  }
  p.out_vec = !odd(p.out, 16) && p.ld_out % 8 == 0;
  p.ws_bf16 = scale_dtype == MOE_BF16;
  p.out_bf16 = out_dtype == MOE_BF16;
  (group == 32   ? launch_w4_group32
   : group == 64 ? launch_w4_group64
                 : launch_w4_group128)(p, workspace, s);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_linear_w4_workspace_bytes(int64_t rows, int32_t experts, int32_t out_features,
                                     int32_t in_features, moe_dtype out_dtype) {
  if (rows <= 0 || rows > kW4Limit || experts <= 0 || experts > kMaxExperts || in_features <= 0 ||
      in_features > kW4Limit || out_features <= 0 || out_features > kW4Limit)
    return 0;
  return w4_workspace(rows, experts, out_features, in_features, out_dtype == MOE_BF16);
}

moe_status moe_linear_w4(const void* x, int64_t ld_x, const uint8_t* w, const void* w_scales,
                         moe_dtype scale_dtype, const uint8_t* w_zeros, const float* bias,
                         int64_t rows, int32_t out_features, int32_t in_features, int32_t group,
                         int32_t swiglu, void* out, int64_t ld_out, moe_dtype out_dtype,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!x || !w || !w_scales || !out) return MOE_ERR_NULL;
  if (swiglu != 0 && swiglu != 1) return MOE_ERR_SHAPE;
  W4Args p{};
  p.x = static_cast<const uint16_t*>(x);
  p.w = w;
  p.ws = w_scales;
  p.wz = w_zeros;
  p.bias = bias;
  p.out = out;
  p.ld_x = ld_x;
  p.ld_out = ld_out;
  p.M = rows;
  p.N = out_features;
  p.K = in_features;
  p.E = 1;
  p.swiglu = swiglu != 0;
  return w4_call(p, group, scale_dtype, out_dtype, workspace, workspace_bytes,
                 static_cast<hipStream_t>(stream));
}

moe_status moe_grouped_linear_w4(const void* x, int64_t ld_x, const int32_t* offsets,
                                 const uint8_t* w, const void* w_scales, moe_dtype scale_dtype,
                                 const uint8_t* w_zeros, const float* bias, int64_t rows,
                                 int32_t experts, int32_t out_features, int32_t in_features,
                                 int32_t group, int32_t swiglu, void* out, int64_t ld_out,
                                 moe_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  if (!x || !offsets || !w || !w_scales || !out) return MOE_ERR_NULL;
  if (swiglu != 0 && swiglu != 1) return MOE_ERR_SHAPE;
  W4Args p{};
  p.x = static_cast<const uint16_t*>(x);
  p.w = w;
  p.ws = w_scales;
  p.wz = w_zeros;
  p.bias = bias;
  p.offsets = offsets;
  p.out = out;
  p.ld_x = ld_x;
  p.ld_out = ld_out;
  p.M = rows;
  p.N = out_features;
  p.K = in_features;
  p.E = experts;
  p.swiglu = swiglu != 0;
  return w4_call(p, group, scale_dtype, out_dtype, workspace, workspace_bytes,
                 static_cast<hipStream_t>(stream));
}

}  // extern "C"
