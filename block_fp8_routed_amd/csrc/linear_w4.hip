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
  bool out_vec;  // eight bf16 values of out from a feature that is a multiple of 8 are aligned
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

// ------------------------------------------------------------ larger batches --
// bf16 output of larger batches: both operands become fp16, so that scale and
// zero point are in the weight itself and the matrix instructions run one chain of
// sums over all of K.
//   x: bf16 has 8 significant bits and fp16 11, so a row times a power of two that
// brings its largest magnitude below 2^15 is exact down to 2^-29 of that magnitude
// (and off by at most 2^-40 of it below). w4_halves writes such rows to the
// workspace, with columns in the order in which codes leave a dword.
//   W: 1024 + q is the fp16 number 0x6400 | q, so (q - z) costs a mask and one
// addition, exact, and its scale one product. The row of weights has a power of two
// that brings its largest scale into [2^6, 2^7) ((q - z) s then stays below 2^15).
// The scale (fp32, or a bf16, which is exact) and the product round once each: at
// most 2^-10 of a term, 3e-4 of the result in norm beside the 1.7e-3 of its
// rounding to bf16. (The exact form takes two fp32 operations on each sum and group.)
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kW4Stage = 128;  // columns of a stage

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
// (1: four rows a workgroup). Rows of up to 512 kHold W columns are read once.
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

// Tile of workgroup b. Workgroups go round-robin over the eight XCDs, each with an
// L2 of its own: XCD x takes a contiguous run of a raster that walks bands of four
// strips of features down the rows.
__device__ __forceinline__ void w4_tile_of(int b, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int total = tiles_m * tiles_n, x = b % kXcdCount, i = b / kXcdCount;
  const int q = total / kXcdCount, r = total % kXcdCount;
  const int t = x * q + (x < r ? x : r) + i;
  constexpr int kBand = 4;
  const int per = kBand * tiles_m, band = t / per, in = t - band * per;
  const int width = tiles_n - band * kBand < kBand ? tiles_n - band * kBand : kBand;
  tm = in / width;
  tn = band * kBand + in - tm * width;
}

// One 16-byte load of each lane into LDS, at lds + 16 lane. An instruction of its
// own: for the builtin the compiler waits for every such load before the next LDS
// read. The stage's wait is w4_wait_loads. It has no register output.
__device__ __forceinline__ void w4_load_lds(uint32_t lds, const void* src) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds), "v"(src)
               : "memory", "m0");
}
__device__ __forceinline__ void w4_wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0f70);
  asm volatile("" ::: "memory");
}

// Eight codes of a dword as (q - z) s in fp16, in the column order of half_order.
// z1 = -(1024 + z), z16 = -(64 + z).
__device__ __forceinline__ f16x8_t codes_f16(uint32_t d, f16x2_t s, f16x2_t z1, f16x2_t z16) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const f16x2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  const uint32_t d8 = d >> 8;
  const auto low = [&](uint32_t v) {
    return (__builtin_bit_cast(f16x2_t, (v & 0x000f000fu) | 0x64006400u) + z1) * s;
  };
  const auto high = [&](uint32_t v) {
    return __builtin_elementwise_fma(__builtin_bit_cast(f16x2_t, (v & 0x00f000f0u) | 0x64006400u),
                                     sixteenth, z16) * s;
  };
  const u32x4 v = {__builtin_bit_cast(uint32_t, low(d)), __builtin_bit_cast(uint32_t, high(d)),
                   __builtin_bit_cast(uint32_t, low(d8)), __builtin_bit_cast(uint32_t, high(d8))};
  return __builtin_bit_cast(f16x8_t, v);
}

// A workgroup of four wavefronts computes 32 FM rows x 256 weight rows; wavefront w
// takes two tiles of 32 weight rows (with swiglu a tile of gates and the tile of
// their ups) and all the rows. A stage is 128 columns: x goes straight to one of two
// LDS buffers, the codes, which only one wavefront needs, to registers; both for
// the next stage while this one is multiplied.
//   An LDS row is 256 bytes; 16-byte piece c of row r lies at c ^ (r & 15), so that
// a fragment's 32 rows reach all banks. Lane l holds columns 64 h .. 64 h + 63 of
// row l % 32 of either operand, h = l / 32; instruction i takes eight of them.
template <int G, int FM>
__global__ __launch_bounds__(256, 2) void w4_tile(W4Args p, const uint16_t* __restrict__ xh,
                                                  const int32_t* __restrict__ xe, int Kp,
                                                  int tiles_m, int tiles_n) {
  constexpr int TM = 32 * FM, kBuf = TM * 256;
  constexpr int NS = G == 32 ? 2 : 1;  // scales of a lane's 64 columns
  __shared__ __attribute__((aligned(1024))) uint8_t ring[2 * kBuf];
  __shared__ int32_t we[4][64];
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int tm, tn;
  w4_tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const RowTile tile = find_tile<TM>(p, tm);
  if (tile.rows <= 0) return;
  const int n_out = p.swiglu ? p.N / 2 : p.N, groups = p.K / G;
  const int n0 = p.swiglu ? tn * 128 + wave * 32 : tn * 256 + wave * 64;
  const int64_t bank = (int64_t)tile.e * p.N;
  const uint8_t* wp[2];
  int64_t sp[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    int n = n0 + l32 + (p.swiglu ? 0 : 32 * j);
    n = (n < n_out ? n : n_out - 1) + (p.swiglu ? j * n_out : 0);
    wp[j] = p.w + (bank + n) * (p.K / 2);
    sp[j] = (bank + n) * groups;
  }
  // x: this thread's pieces of a stage, rows 16 apart (which leaves the swizzle alone)
  const int r0 = tid >> 4;
  const uint16_t* xp[2 * FM];
#pragma unroll
  for (int i = 0; i < 2 * FM; ++i) {
    const int r = r0 + 16 * i < tile.rows ? r0 + 16 * i : tile.rows - 1;
    xp[i] = xh + (tile.r0 + r) * Kp + 8 * ((tid & 15) ^ r0);
  }
  const uint32_t lds0 =
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)ring + 1024 * wave;
  const auto issue = [&](int kb) {
#pragma unroll
    for (int i = 0; i < 2 * FM; ++i)
      w4_load_lds(lds0 + (kb & 1) * kBuf + 4096 * i, xp[i] + kb * kW4Stage);
  };
  struct Codes {
    uint4 v[2][2];
    float s[2][NS], z[2][NS];
  };
  const auto fetch = [&](int kb) {
    Codes c;
    const int col = kb * kW4Stage + 64 * h;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 0; i < 2; ++i)  // (x is zero behind K: any code will do)
        c.v[j][i] = ld16(wp[j] + (col + 32 * i < p.K ? col + 32 * i : 0) / 2);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int g = col / G + i < groups ? col / G + i : groups - 1;
        c.s[j][i] = p.ws_bf16 ? bf16_lo(static_cast<const uint16_t*>(p.ws)[sp[j] + g])
                              : static_cast<const float*>(p.ws)[sp[j] + g];
        c.z[j][i] = p.wz ? (float)p.wz[sp[j] + g] : 8.f;
      }
    }
    return c;
  };
  issue(0);
  Codes next = fetch(0);
  // the weight rows' powers of two
  int en[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float m = 0.f;
#pragma unroll 4
    for (int g = h; g < groups; g += 2)
      m = fmaxf(m, fabsf(p.ws_bf16 ? bf16_lo(static_cast<const uint16_t*>(p.ws)[sp[j] + g])
                                   : static_cast<const float*>(p.ws)[sp[j] + g]));
    m = fmaxf(m, __shfl_xor(m, 32));
    en[j] = m > 0.f ? __builtin_amdgcn_frexp_expf(m) - 7 : 0;
    if (h == 0) we[wave][32 * j + l32] = en[j];
  }
  f32x16 acc[2][FM];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[j][m][v] = 0.f;
  const int stages = Kp / kW4Stage;
#pragma unroll 1
  for (int kb = 0; kb < stages; ++kb) {
    w4_wait_loads();
    lds_barrier();  // everyone's pieces are there, and the other buffer has been read
    const Codes c = next;
    if (kb + 1 < stages) {
      issue(kb + 1);
      next = fetch(kb + 1);
    }
    f16x2_t s[2][NS], z1[2][NS], z16[2][NS];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const _Float16 sv = (_Float16)__builtin_ldexpf(c.s[j][i], -en[j]);
        const _Float16 a = (_Float16)(-1024.f - c.z[j][i]), b = (_Float16)(-64.f - c.z[j][i]);
        s[j][i] = f16x2_t{sv, sv};
        z1[j][i] = f16x2_t{a, a};
        z16[j][i] = f16x2_t{b, b};
      }
    const uint8_t* buf = ring + (kb & 1) * kBuf + l32 * 256;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f16x8_t x[FM], w[2];
#pragma unroll
      for (int m = 0; m < FM; ++m)
        x[m] = __builtin_bit_cast(
            f16x8_t, *reinterpret_cast<const uint4*>(buf + m * 8192 + 16 * ((8 * h + i) ^ (l32 & 15))));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 q = c.v[j][i / 4];
        const uint32_t d[4] = {q.x, q.y, q.z, q.w};
        constexpr int kPer = 8 / NS;
        w[j] = codes_f16(d[i % 4], s[j][i / kPer], z1[j][i / kPer], z16[j][i / kPer]);
      }
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[j][m] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w[j], x[m], acc[j][m], 0, 0, 0);
    }
  }
  // Value v of a lane: weight row 8 (v / 4) + 4 h + v % 4, row l32 of x. Rows go out
  // through LDS (the ring is free) in 16-byte pieces: a lane's four features are
  // half a piece.
  lds_barrier();
  const int width = p.swiglu ? 64 : 128;  // bytes of a wavefront's output row
  uint8_t* mine = ring + wave * (TM * 128);
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int r = 32 * m + l32;
    const int er = xe[tile.r0 + (r < tile.rows ? r : tile.rows - 1)];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int f = 8 * b + 4 * h;
      float y[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int4 e4 = *reinterpret_cast<const int4*>(&we[wave][32 * j + f]);
        const int e[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          y[j][v] = __builtin_ldexpf(acc[j][m][4 * b + v], e[v] + er);
          if (p.bias) {
            int n = n0 + f + v + (p.swiglu ? 0 : 32 * j);
            n = (n < n_out ? n : n_out - 1) + (p.swiglu ? j * n_out : 0);
            y[j][v] += p.bias[bank + n];
          }
        }
      }
      const auto put = [&](int piece, const float (&v)[4]) {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<bf16x4*>(mine + r * width + 16 * piece + 8 * h) =
            bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
      };
      if (p.swiglu) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = y[0][i] / (1.f + expf(-y[0][i])) * y[1][i];
        put(b ^ ((r >> 1) & 3), v);
      } else {
        put(b ^ (r & 7), y[0]);
        put((4 + b) ^ (r & 7), y[1]);
      }
    }
  }
  wave_lds_fence();
  const int per = width / 16;  // pieces a row
  uint16_t* out = static_cast<uint16_t*>(p.out);
  for (int i = lane; i < TM * per; i += 64) {
    const int r = i / per, c = i % per, n = n0 + 8 * c;
    if (r >= tile.rows) break;
    const uint4 v = *reinterpret_cast<const uint4*>(
        mine + r * width + 16 * (p.swiglu ? c ^ ((r >> 1) & 3) : c ^ (r & 7)));
    uint16_t* at = out + (tile.r0 + r) * p.ld_out + n;
    if (p.out_vec && n + 8 <= n_out) {
      *reinterpret_cast<uint4*>(at) = v;
    } else {
      const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (n + k < n_out) at[k] = (uint16_t)(d[k / 2] >> (16 * (k & 1)));
    }
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

static size_t al256(size_t n) { return (n + 255) / 256 * 256; }
static int padded(int K) { return (K + kW4Stage - 1) / kW4Stage * kW4Stage; }

// Whether a product takes the fp16 tiles.
static bool takes_tiles(int64_t M, int E, moe_dtype out_dtype) {
  return out_dtype == MOE_BF16 && M > 64 * (int64_t)E;
}

static size_t w4_workspace(int64_t M, int E, int K, moe_dtype out_dtype) {
  if (!takes_tiles(M, E, out_dtype)) return 0;
  return al256((size_t)M * padded(K) * 2) + al256((size_t)M * 4);
}

template <int G, int FM>
static void launch_w4_tile(const W4Args& p, const uint16_t* xh, const int32_t* xe, hipStream_t s) {
  const int n_out = p.swiglu ? p.N / 2 : p.N, cols = p.swiglu ? 128 : 256;
  const int tm = (int)row_tiles(p, 32 * FM), tn = (n_out + cols - 1) / cols;
  w4_tile<G, FM><<<(unsigned)((int64_t)tm * tn), 256, 0, s>>>(p, xh, xe, padded(p.K), tm, tn);
}

template <int G>
static void launch_w4(const W4Args& p, void* workspace, hipStream_t s) {
  if (takes_tiles(p.M, p.E, p.out_bf16 ? MOE_BF16 : MOE_F32)) {
    const int Kp = padded(p.K);
    uint4* xh = static_cast<uint4*>(workspace);
    int32_t* xe = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) +
                                             al256((size_t)p.M * Kp * 2));
    if (p.K <= 2048)
      w4_halves<1><<<(unsigned)((p.M + 3) / 4), 256, 0, s>>>(p.x, p.ld_x, p.M, p.K, Kp, xh, xe);
    else
      w4_halves<4><<<(unsigned)p.M, 256, 0, s>>>(p.x, p.ld_x, p.M, p.K, Kp, xh, xe);
    launch_w4_tile<G, 4>(p, reinterpret_cast<const uint16_t*>(xh), xe, s);
    return;
  }
  launch_w4_rows<G, 1, 2, 8>(p, s);
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
  // fewer than 2^32 threads a grid: 512 a workgroup of 16 rows and 16 features
  if (row_tiles(p, 16) * ((p.N + 15) / 16) >= ((int64_t)1 << 23)) return MOE_ERR_UNSUPPORTED;
  if (p.M == 0) return MOE_OK;
  const auto odd = [](const void* q, int n) { return reinterpret_cast<uintptr_t>(q) % n != 0; };
  if (odd(p.x, 16) || odd(p.w, 16) || p.ld_x % 8 != 0 || odd(p.ws, scale_dtype == MOE_BF16 ? 2 : 4) ||
      odd(p.bias, 4) || odd(p.offsets, 4) || odd(p.out, out_dtype == MOE_BF16 ? 2 : 4))
    return MOE_ERR_UNSUPPORTED;
  const size_t need = w4_workspace(p.M, p.E, p.K, out_dtype);
  if (need > 0) {
    if (!workspace) return MOE_ERR_NULL;
    if (workspace_bytes < need || odd(workspace, 256)) return MOE_ERR_WORKSPACE;
  }
  p.out_vec = !odd(p.out, 16) && p.ld_out % 8 == 0;
  p.ws_bf16 = scale_dtype == MOE_BF16;
  p.out_bf16 = out_dtype == MOE_BF16;
  if (group == 32)
    launch_w4<32>(p, workspace, s);
  else if (group == 64)
    launch_w4<64>(p, workspace, s);
  else
    launch_w4<128>(p, workspace, s);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_linear_w4_workspace_bytes(int64_t rows, int32_t experts, int32_t in_features,
                                     moe_dtype out_dtype) {
  if (rows <= 0 || rows > kW4Limit || experts <= 0 || experts > kMaxExperts || in_features <= 0 ||
      in_features > kW4Limit)
    return 0;
  return w4_workspace(rows, experts, in_features, out_dtype);
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
