// linear_w4.hip — moe_linear_w4 and moe_grouped_linear_w4: products with 4-bit
// weights,
//   out[t][n] = sum_k x[t][k] (q[n][k] - z[n][g]) s[n][g] (+ bias[n]),  g = k / G,
// one bank for all rows, or one bank an expert for rows sorted by expert.
//
// A group's sum is split as s (sum_k x q - z sum_k x): the matrix instruction
// multiplies bf16 rows of x with the codes themselves, which bf16 holds exactly,
// and fp32 takes scale and zero point. Nothing is rounded before the output.
// The codes get to bf16 as E4M3 bytes: byte q (0 .. 15) is the E4M3 number q 2^-9
// (0 .. 7 are its subnormals, 8 .. 15 its first binade), so a masked nibble is
// already an operand of the conversion instruction. The factor 2^9 goes into s.
#include "device.hpp"
#include "layer.hpp"

namespace moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

struct W4Args {
  const uint16_t* x;       // [M] rows of K bf16, ld_x apart
  const uint8_t* w;        // [E][N][K/2], the even column in a byte's low half
  const void* ws;          // [E][N][K/G] fp32 or bf16
  const uint8_t* wz;       // [E][N][K/G] or null: 8
  const float* bias;       // [E][N] or null
  const int32_t* offsets;  // [E+1] first rows, or null: all rows are expert 0's
  void* out;
  int64_t ld_x, ld_out, M;
  int N, K, E;
  bool ws_bf16, out_bf16, swiglu;
};

// Rows [r0, r0 + rows) of expert e; rows = 0: none.
struct RowTile {
  int e, rows;
  int64_t r0;
};

// The slot-th tile of at most TM rows. Experts' tiles follow each other; lane l
// counts those of experts [l c, (l + 1) c), a scan finds the lane whose tiles hold
// the slot, and that lane's experts are walked. Offsets are cut to [0, M].
template <int TM>
__device__ __forceinline__ RowTile find_tile(const W4Args& p, int slot) {
  RowTile r;
  if (!p.offsets) {
    r.e = 0;
    r.r0 = (int64_t)slot * TM;
    const int64_t left = p.M - r.r0;
    r.rows = left < TM ? (int)left : TM;
    return r;
  }
  const int lane = threadIdx.x & 63;
  const int c = (p.E + 63) / 64, e0 = lane * c;
  const int M = (int)p.M;
  const auto at = [&](int e) {
    const int v = p.offsets[e < p.E ? e : p.E];
    return v < 0 ? 0 : v > M ? M : v;
  };
  int tiles = 0, last = at(e0);
  for (int i = 1; i <= c; ++i) {
    const int next = at(e0 + i);
    if (next > last) tiles += (next - last + TM - 1) / TM;
    last = next;
  }
  const int incl = wave_incl_scan(tiles);
  const uint64_t past = __ballot(incl > slot);
  r.e = 0;
  r.r0 = 0;
  r.rows = 0;
  if (past == 0) return r;
  const int owner = __builtin_ctzll(past);
  int left = slot - (__builtin_amdgcn_readlane(incl, owner) - __builtin_amdgcn_readlane(tiles, owner));
  for (int e = owner * c; e < owner * c + c; ++e) {
    const int lo = at(e), hi = at(e + 1);
    if (hi <= lo) continue;
    const int n = (hi - lo + TM - 1) / TM;
    if (left < n) {
      r.e = e;
      r.r0 = lo + left * TM;
      r.rows = hi - (int)r.r0 < TM ? hi - (int)r.r0 : TM;
      break;
    }
    left -= n;
  }
  r.e = __builtin_amdgcn_readfirstlane(r.e);
  r.rows = __builtin_amdgcn_readfirstlane(r.rows);
  r.r0 = __builtin_amdgcn_readfirstlane((int)r.r0);
  return r;
}

// Eight codes of a dword as bf16 (times 2^-9), in the column order 0 2 4 6 1 3 5 7.
__device__ __forceinline__ bf16x8_t codes_bf16(uint32_t d) {
  const uint32_t even = d & 0x0f0f0f0fu, odd = (d >> 4) & 0x0f0f0f0fu;
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 v = {__builtin_bit_cast(uint32_t, e4m3x2_to_bf16x2<false>(even)),
                   __builtin_bit_cast(uint32_t, e4m3x2_to_bf16x2<true>(even)),
                   __builtin_bit_cast(uint32_t, e4m3x2_to_bf16x2<false>(odd)),
                   __builtin_bit_cast(uint32_t, e4m3x2_to_bf16x2<true>(odd))};
  return __builtin_bit_cast(bf16x8_t, v);
}
// Eight bf16 values of x brought to that order.
__device__ __forceinline__ bf16x8_t x_order(uint4 v) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 o = {__builtin_amdgcn_perm(v.y, v.x, 0x05040100u),
                   __builtin_amdgcn_perm(v.w, v.z, 0x05040100u),
                   __builtin_amdgcn_perm(v.y, v.x, 0x07060302u),
                   __builtin_amdgcn_perm(v.w, v.z, 0x07060302u)};
  return __builtin_bit_cast(bf16x8_t, o);
}

// Lane quarter q holds dwords 0 .. 3 of block q; leaves dword q of blocks 0 .. 3.
__device__ __forceinline__ void transpose_quarters(uint4& v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  v = make_uint4(c[0], c[1], d[0], d[1]);
}

constexpr float kCodeScale = 512.f;  // 2^9: a code's operand is q 2^-9

__device__ __forceinline__ float w4_scale(const W4Args& p, int64_t i) {
  const float s = p.ws_bf16 ? bf16_lo(static_cast<const uint16_t*>(p.ws)[i])
                            : static_cast<const float*>(p.ws)[i];
  return s * kCodeScale;
}

__device__ __forceinline__ void w4_store(const W4Args& p, int64_t row, int n, float v) {
  if (p.out_bf16)
    static_cast<__bf16*>(p.out)[row * p.ld_out + n] = (__bf16)v;
  else
    static_cast<float*>(p.out)[row * p.ld_out + n] = v;
}

// Few rows: W wavefronts share 16 FN weight rows and 16 FM rows of x, and split K
// by units of 128 columns; their sums are joined in LDS in wavefront order.
// Lane l reads 16 bytes (32 codes) of weight row l % 16 at quarter l / 16 of the
// unit; after the exchange between the quarters instruction b covers the unit's
// columns 32 b .. 32 b + 31, so that every group size is a whole number of
// instructions. x is the A operand: a lane ends with four rows of one output
// feature, whose scale it holds itself. The sums of x come from the same
// instruction, with ones (2^-9) for the weights.
template <int G, int FM, int FN, int W>
__global__ __launch_bounds__(64 * W) void w4_rows(W4Args p) {
  constexpr int TM = 16 * FM;
  __shared__ float part[W][FM][FN][4][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, l = lane & 15, q = lane >> 4;
  const int n_out = p.swiglu ? p.N / 2 : p.N, cols = p.swiglu ? 8 * FN : 16 * FN;
  const int strips = (n_out + cols - 1) / cols;
  const RowTile tile = find_tile<TM>(p, blockIdx.x / strips);
  if (tile.rows <= 0) return;
  const int n0 = (int)(blockIdx.x % strips) * cols;
  const int64_t bank = (int64_t)tile.e * p.N;
  const int groups = p.K / G;
  // this lane's weight row of each tile (rows past the last repeat it)
  const uint8_t* wp[FN];
  int64_t sp[FN];
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    int n = p.swiglu && FN > 1 ? n0 + 16 * (f % (FN / 2 > 0 ? FN / 2 : 1)) + l : n0 + 16 * f + l;
    if (n >= n_out) n = n_out - 1;
    if (p.swiglu && f >= FN / 2) n += n_out;
    wp[f] = p.w + (bank + n) * (p.K / 2);
    sp[f] = (bank + n) * groups;
  }
  const uint16_t* xp[FM];
#pragma unroll
  for (int f = 0; f < FM; ++f) {
    const int r = 16 * f + l < tile.rows ? 16 * f + l : tile.rows - 1;
    xp[f] = p.x + (tile.r0 + r) * p.ld_x;
  }
  bf16x8_t ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)(1.f / kCodeScale);
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int f = 0; f < FN; ++f) acc[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int k0 = 128 * w; k0 < p.K; k0 += 128 * W) {
    uint4 code[FN];
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      code[f] = make_uint4(0, 0, 0, 0);
      if (k0 + 32 * q < p.K) code[f] = ld16(wp[f] + (k0 + 32 * q) / 2);
    }
    uint4 xv[4][FM];
#pragma unroll
    for (int b = 0; b < 4; ++b)
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        xv[b][i] = make_uint4(0, 0, 0, 0);
        if (k0 + 32 * b < p.K) xv[b][i] = ld16(xp[i] + k0 + 32 * b + 8 * q);
      }
    constexpr int NG = 128 / G, NB = G / 32;  // groups of the unit, instructions of a group
    float s[NG][FN], z[NG][FN];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int at = k0 / G + g < groups ? k0 / G + g : groups - 1;
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        s[g][f] = w4_scale(p, sp[f] + at);
        z[g][f] = p.wz ? (float)p.wz[sp[f] + at] : 8.f;
      }
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) transpose_quarters(code[f]);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x4 d[FM][FN], xs[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        xs[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < FN; ++f) d[i][f] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int b = g * NB; b < (g + 1) * NB; ++b) {
        bf16x8_t a[FM];
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          a[i] = x_order(xv[b][i]);
          xs[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], ones, xs[i], 0, 0, 0);
        }
#pragma unroll
        for (int f = 0; f < FN; ++f) {
          const uint32_t cw[4] = {code[f].x, code[f].y, code[f].z, code[f].w};
          const bf16x8_t bw = codes_bf16(cw[b]);
#pragma unroll
          for (int i = 0; i < FM; ++i)
            d[i][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], bw, d[i][f], 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[i][f][v] = fmaf(s[g][f], fmaf(-z[g][f], xs[i][v], d[i][f][v]), acc[i][f][v]);
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
      for (int v = 0; v < 4; ++v) part[w][i][f][v][lane] = acc[i][f][v];
  __syncthreads();
  // value (row 16 i + r, feature 16 f + c) lies at lane 16 (r / 4) + c, v = r % 4
  const auto total = [&](int i, int f, int r, int c) {
    float y = 0.f;
#pragma unroll
    for (int ww = 0; ww < W; ++ww) y += part[ww][i][f][r & 3][16 * (r >> 2) + c];
    return y;
  };
  for (int i = threadIdx.x; i < TM * cols; i += 64 * W) {
    const int r = i / cols, c = i % cols, n = n0 + c;
    if (r >= tile.rows || n >= n_out) continue;
    float y = total(r / 16, c / 16, r % 16, c % 16);
    if (p.bias) y += p.bias[bank + n];
    if (p.swiglu) {
      float u = total(r / 16, FN / 2 + c / 16, r % 16, c % 16);
      if (p.bias) u += p.bias[bank + n_out + n];
      y = y / (1.f + expf(-y)) * u;
    }
    w4_store(p, tile.r0 + r, n, y);
  }
}

// ---------------------------------------------------------------- host side --
// Row tiles of at most TM rows: every expert's last one may be short.
static int64_t row_tiles(const W4Args& p, int TM) {
  return p.offsets ? p.M / TM + (p.M < p.E ? p.M : p.E) : (p.M + TM - 1) / TM;
}

template <int G, int FM, int FN, int W>
static void launch_w4_rows(const W4Args& p, hipStream_t s) {
  const int n_out = p.swiglu ? p.N / 2 : p.N, cols = p.swiglu ? 8 * FN : 16 * FN;
  w4_rows<G, FM, FN, W><<<(unsigned)(row_tiles(p, 16 * FM) * ((n_out + cols - 1) / cols)), 64 * W,
                         0, s>>>(p);
}

template <int G>
static void launch_w4(const W4Args& p, hipStream_t s) {
  launch_w4_rows<G, 1, 2, 8>(p, s);
}

static moe_status w4_call(W4Args p, int group, moe_dtype scale_dtype, moe_dtype out_dtype,
                          hipStream_t s) {
  if (p.M < 0 || p.N <= 0 || p.K <= 0 || p.E <= 0 || group <= 0) return MOE_ERR_SHAPE;
  if (p.K % group != 0 || (p.swiglu && p.N % 2 != 0)) return MOE_ERR_SHAPE;
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return MOE_ERR_SHAPE;
  if (scale_dtype != MOE_F32 && scale_dtype != MOE_BF16) return MOE_ERR_SHAPE;
  if (p.ld_x < p.K || p.ld_out < (p.swiglu ? p.N / 2 : p.N)) return MOE_ERR_SHAPE;
  if (group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
  if (p.E > kMaxExperts || p.K > (1 << 20) || p.N > (1 << 20) || p.M > (1 << 20))
    return MOE_ERR_UNSUPPORTED;
  // fewer than 2^32 threads a grid: 512 a workgroup of 16 rows and 16 features
  if (row_tiles(p, 16) * ((p.N + 15) / 16) >= ((int64_t)1 << 23)) return MOE_ERR_UNSUPPORTED;
  if (p.M == 0) return MOE_OK;
  const auto odd = [](const void* q, int n) { return reinterpret_cast<uintptr_t>(q) % n != 0; };
  if (odd(p.x, 16) || odd(p.w, 16) || p.ld_x % 8 != 0 || odd(p.ws, scale_dtype == MOE_BF16 ? 2 : 4) ||
      odd(p.bias, 4) || odd(p.offsets, 4) || odd(p.out, out_dtype == MOE_BF16 ? 2 : 4))
    return MOE_ERR_UNSUPPORTED;
  p.ws_bf16 = scale_dtype == MOE_BF16;
  p.out_bf16 = out_dtype == MOE_BF16;
  if (group == 32)
    launch_w4<32>(p, s);
  else if (group == 64)
    launch_w4<64>(p, s);
  else
    launch_w4<128>(p, s);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_linear_w4(const void* x, int64_t ld_x, const uint8_t* w, const void* w_scales,
                         moe_dtype scale_dtype, const uint8_t* w_zeros, const float* bias,
                         int64_t rows, int32_t out_features, int32_t in_features, int32_t group,
                         int32_t swiglu, void* out, int64_t ld_out, moe_dtype out_dtype,
                         void* stream) {
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
  return w4_call(p, group, scale_dtype, out_dtype, static_cast<hipStream_t>(stream));
}

moe_status moe_grouped_linear_w4(const void* x, int64_t ld_x, const int32_t* offsets,
                                 const uint8_t* w, const void* w_scales, moe_dtype scale_dtype,
                                 const uint8_t* w_zeros, const float* bias, int64_t rows,
                                 int32_t experts, int32_t out_features, int32_t in_features,
                                 int32_t group, int32_t swiglu, void* out, int64_t ld_out,
                                 moe_dtype out_dtype, void* stream) {
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
  return w4_call(p, group, scale_dtype, out_dtype, static_cast<hipStream_t>(stream));
}

}  // extern "C"
