// linear.hip — moe_linear and moe_linear_e4m3: one dense product with
// block-FP8 weights and E4M3 activations,
//   out[t][n] = sum_kb s[n/128][kb] * sum_{k in kb} a[t][k] * dec(w[n][k]) (+ bias[n]).
//
// bf16 output of the tile kernels: the inner sum of one 128-column block is one
// matrix instruction (v_mfma_scale_f32_16x16x128_f8f6f4) over 16 weight rows and 16
// activation rows. The activations' power-of-two scale is the instruction's
// own E8M0 scale; the weights' fp32 block scale, which is no power of two,
// multiplies the instruction's fp32 result as it is added to the running sum.
// The instruction sums eight consecutive products of a lane on one grid, 2^-13
// of the largest (measured: 2^16 + 2^3 is exact, 2^16 + 2^2 loses the second
// term), so a sum errs by at most 2^-10 of its terms' magnitudes. Towards zero, the
// cuts of terms of either sign go either way: 6e-5 of the result in norm (measured
// at K = 512 and 1024), where the output's rounding is 1.7e-3. An element whose
// terms cancel has no bound relative to itself.
//
// (What follows may see the cuts through its own rounding: a bf16 value or an
// E4M3 code near a midpoint falls to either side. The exact form below would take
// 535 us where this one takes 240 to 260; fp32 output is the caller's way to it.)
//
// fp32 output: that error would be the result's, so the codes are widened to
// fp16 in registers (exact) and go through v_mfma_f32_16x16x32_f16, which
// keeps 2^-24 of the largest of eight products; the activations' scale is
// applied to the instruction's result. Small batches take this form for both
// output types. Its conversions bound the large tiles: 96 of them and 32 matrix
// instructions a stage of 32 x 64 outputs (8192 x 8192 x 4096: 1030 TFLOP/s). A
// single round of 128 x 128 tiles has some 8 us that do not go with K (16.5 us at
// K = 1024, 41 at 4096): its ring holds one stage ahead.
//
// Weights are the instruction's A operand, so that a lane ends with four
// consecutive output features of one row.
#include "device.hpp"
#include "e4m3_round.hpp"
#include "layer.hpp"

namespace moe {

constexpr int kLinB = 128;  // columns per scale block

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct LinearArgs {
  const uint16_t* x;     // [M] rows of K bf16, ld_x apart, or null: codes and exps
  int64_t ld_x;
  const uint8_t* codes;  // [M][K]
  const uint8_t* exps;   // [M][K/128]
  const uint8_t* w;      // [N][K]
  const float* ws;       // [ceil(N/128)][K/128]
  const float* bias;     // [N] or null
  void* out;
  int64_t M, ld_out;
  int N, K;
  bool vec4;  // four values of out from a feature that is a multiple of 4 are aligned
  bool vec8;  // likewise eight bf16 values, to 16 bytes
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

// One block's share acc += s * 2^(scale - 127) * (A B over 128 k), in two
// steps: block_product (the matrix instructions) and add_block (scales and
// sum). Lane l holds row l % 16 of each operand and the 32 k of its quarter
// l / 16 (any 32, the same for both operands); the result's column l % 16 (B's
// row) at rows 4 (l / 16) + v. Byte SEL of scale is the E8M0 byte of B's row;
// s is the weights' block scale, premultiplied as block_scale() does.
// The sums must neither overflow nor fall below what fp32 holds before s joins. With
// codes and exponents as the quantisers write them (codes of 256 at most at the
// exponent 120, which takes the ends of bf16 and fp32; 448 below) a sum of 128
// products stays below 2^143.81, so the FP8 instruction's A operand has the
// constant scale 2^-kHold: 2^127.81. At the other end each of its sixteen groups of
// products is then cut at 2^-149, where the smallest product of a block of exponent
// e is 2^-18 2^(e - kHold): below e = -115 a block may lose 2^-145 2^kHold s. The
// fp16 form takes what is above 2^100 out of 2^e and loses nothing (2^-18 2^-127
// is a subnormal fp32 value, and kept).
constexpr int kHold = 16;
template <bool BF16>
__device__ __forceinline__ float block_scale(float s) {
  return BF16 ? s * (float)(1 << kHold) : s;
}
template <bool BF16, int SEL>
__device__ __forceinline__ f32x4 block_product(const i32x8_t& a, const i32x8_t& b, int scale) {
  f32x4 d = {0.f, 0.f, 0.f, 0.f};
  if (BF16)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, d, 0, 0, 0, 127 - kHold, SEL,
                                                            scale);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    d = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(a[2 * j], a[2 * j + 1]),
                                               widen(b[2 * j], b[2 * j + 1]), d, 0, 0, 0);
  return d;
}
template <bool BF16>
__device__ __forceinline__ f32x4 block_product_sel(const i32x8_t& a, const i32x8_t& b, int scale,
                                                   int sel) {  // sel: a constant once unrolled
  switch (sel) {
    case 0: return block_product<BF16, 0>(a, b, scale);
    case 1: return block_product<BF16, 1>(a, b, scale);
    case 2: return block_product<BF16, 2>(a, b, scale);
    default: return block_product<BF16, 3>(a, b, scale);
  }
}
template <bool BF16>
__device__ __forceinline__ void add_block(f32x4& acc, const f32x4& d, int scale, int sel, float s) {
  if (BF16) {
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = fmaf(s, d[v], acc[v]);
    return;
  }
  const int e = (int)(((uint32_t)scale >> (8 * sel)) & 255u) - 127, e0 = e < 100 ? e : 100;
  const float se = __builtin_ldexpf(s, e - e0);
#pragma unroll
  for (int v = 0; v < 4; ++v) acc[v] = fmaf(se, __builtin_ldexpf(d[v], e0), acc[v]);
}

// One byte, or an aligned dword, of a buffer (0 past its range).
__device__ __forceinline__ uint32_t buffer_ld1(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0);
}
__device__ __forceinline__ uint32_t buffer_ld4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
}

// Keeps what uses v behind what stands before (no instruction).
__device__ __forceinline__ void pin(f32x4& v) { asm volatile("" : "+v"(v)); }

template <bool BF16>
__device__ __forceinline__ void store_out(void* out, int64_t at, float v) {
  if (BF16)
    reinterpret_cast<uint16_t*>(out)[at] = (uint16_t)f32_to_bf16_bits(v);
  else
    reinterpret_cast<float*>(out)[at] = v;
}

// Four consecutive features n .. n + 3 of one row (fewer at the end of N).
template <bool BF16>
__device__ __forceinline__ void store4(const LinearArgs& p, int64_t row, int n, f32x4 v) {
  if (n >= p.N) return;
  if (p.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] += p.bias[n + j < p.N ? n + j : p.N - 1];
  }
  const int64_t at = row * p.ld_out + n;
  if (p.vec4 && n + 4 <= p.N) {
    if (BF16)
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + at) =
          make_uint2(f32_to_bf16_bits(v[0]) | f32_to_bf16_bits(v[1]) << 16,
                     f32_to_bf16_bits(v[2]) | f32_to_bf16_bits(v[3]) << 16);
    else
      *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p.out) + at) = v;
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (n + j < p.N) store_out<BF16>(p.out, at + j, v[j]);
}

// Tile of workgroup b. Workgroups go round-robin over the eight XCDs, each
// with an L2 of its own: XCD x takes a contiguous run of a raster that walks
// bands of four feature tiles down the rows, so that the workgroups it runs
// together share operands.
__device__ __forceinline__ void linear_tile_of(int b, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int total = tiles_m * tiles_n, x = b % kXcdCount, i = b / kXcdCount;
  const int q = total / kXcdCount, r = total % kXcdCount;
  const int t = x * q + (x < r ? x : r) + i;
  constexpr int kBand = 4;
  const int per = kBand * tiles_m, band = t / per, in = t - band * per;
  const int width = tiles_n - band * kBand < kBand ? tiles_n - band * kBand : kBand;
  tm = in / width;
  tn = band * kBand + in - tm * width;
}

// Small batches: the weights' bytes bound the product, so it is laid out as a
// stream of them. A workgroup takes 16 FN output features and up to 16 FM
// rows; its W wavefronts take every W-th block of K, U blocks requested
// together; the partial sums meet in LDS and are added in wavefront order. The
// products are the exact fp16 ones for both output types: the matrix units
// have room to spare here.
//   A load covers whole 128-byte lines (eight rows of codes, four of bf16). The
// matrix instruction wants 16 rows and a quarter of the columns in each
// wavefront's quarter instead, so a wavefront passes its blocks through LDS of
// its own. Loads straight in that form, half lines of 16 rows, take 28 B/ns into a
// compute unit, whatever hangs on them (77 x 2112 x 4096: 11.4 us; so 7.9; with
// the exchange left out 7.3).
//   XQ: the activations are bf16 rows of x, quantised as they are read: a
// lane holds 32 of a row's 128 columns, the row's four lanes agree on the
// largest magnitude, and the conversion instruction does the rest.
__device__ __forceinline__ i32x8_t quantised_operand(const uint4 (&v)[4], int& e) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, bf16x8_max_abs(v[i]));
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  e = act_exponent(__uint_as_float(m << 16));
  i32x8_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint2 q = e4m3x8_of_bf16(v[i], e);
    o[2 * i] = (int)q.x;
    o[2 * i + 1] = (int)q.y;
  }
  e += 127;
  return o;
}

template <int FM, int FN, int W, int U, bool XQ, bool BF16>
__device__ __forceinline__ void linear_rows_body(const LinearArgs& p) {
  constexpr int AL = XQ ? 4 : 2;  // loads of a fragment of activations
  constexpr int kWave = 1024 * (FM * AL + FN * 2);
  static_assert(kWave >= 1024 * FM * FN, "partial sums take the blocks' place");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[W * kWave];
  const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const mine = lds + wave * kWave;
  const int n0 = blockIdx.x * 16 * FN;
  const int64_t m0 = (int64_t)blockIdx.y * 16 * FM;
  const int KB = p.K / kLinB;
  // load j of a fragment: rows 8 j + lane / 8, 16-byte piece lane % 8
  const uint8_t* wp[FN][2];
  const float* sp[FN];
#pragma unroll
  for (int n = 0; n < FN; ++n) {
    const int nt = n0 + 16 * n < p.N ? n0 + 16 * n : n0;  // a tile past the end repeats the first
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = nt + 8 * j + (lane >> 3) < p.N ? nt + 8 * j + (lane >> 3) : p.N - 1;
      wp[n][j] = p.w + (size_t)r * p.K + 16 * (lane & 7);
    }
    sp[n] = p.ws + (size_t)(nt / kLinB) * KB;
  }
  // (bf16: rows 4 j + lane / 16, piece lane % 16)
  const uint8_t* ap[FM][AL];
  const uint8_t* ep[FM];
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int64_t t = m0 + 16 * m, last = p.M - 1;
#pragma unroll
    for (int j = 0; j < AL; ++j) {
      const int64_t r = XQ ? t + 4 * j + q : t + 8 * j + (lane >> 3);
      if (XQ)
        ap[m][j] = reinterpret_cast<const uint8_t*>(p.x + (r < last ? r : last) * p.ld_x + 8 * l16);
      else
        ap[m][j] = p.codes + (size_t)(r < last ? r : last) * p.K + 16 * (lane & 7);
    }
    if (!XQ) ep[m] = p.exps + (size_t)(t + l16 < last ? t + l16 : last) * KB;
  }
  // Piece c of row r is at slot c ^ (r / 2 % 8) of the row's 128 bytes, or
  // c ^ r % 16 of its 256: both sides of the exchange reach all banks.
  const int r8 = lane >> 3;
  const int put8 = 128 * r8 + 16 * ((lane & 7) ^ (r8 >> 1));   // j: + 1024 j, piece ^ 4 j
  const int get8 = 128 * l16 + 16 * (q ^ (l16 >> 1));          // second half: piece ^ 4
  f32x4 acc[FN][FM];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[n][m] = f32x4{0.f, 0.f, 0.f, 0.f};

  // U blocks a round; blocks past the end repeat the last one with scale 0
  for (int kb0 = wave; kb0 < KB; kb0 += W * U) {
    uint4 w[U][FN][2], av[U][FM][AL];
    int ev[U][FM];
    float s[U][FN];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k0 = kb0 + u * W, kb = k0 < KB ? k0 : KB - 1;
#pragma unroll
      for (int n = 0; n < FN; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) w[u][n][j] = ld16(wp[n][j] + (size_t)kb * kLinB);
        s[u][n] = k0 < KB ? sp[n][kb] : 0.f;
      }
#pragma unroll
      for (int m = 0; m < FM; ++m) {
#pragma unroll
        for (int j = 0; j < AL; ++j)
          av[u][m][j] = ld16(ap[m][j] + (size_t)kb * (XQ ? 2 * kLinB : kLinB));
        if (!XQ) ev[u][m] = ep[m][kb];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const auto store = [&](int at, uint4 v) { *reinterpret_cast<uint4*>(mine + at) = v; };
      const auto fetch = [&](int at) { return *reinterpret_cast<const uint4*>(mine + at); };
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) store(2048 * n + 1024 * j + (put8 ^ 64 * j), w[u][n][j]);
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int j = 0; j < AL; ++j)
          store(2048 * FN + 1024 * (AL * m + j) +
                    (XQ ? 256 * q + 16 * (l16 ^ (4 * j + q)) : put8 ^ 64 * j),
                av[u][m][j]);
      wave_lds_fence();
      i32x8_t b[FN], a[FM];
      int e[FM];
#pragma unroll
      for (int n = 0; n < FN; ++n)
        b[n] = operand(fetch(2048 * n + get8), fetch(2048 * n + (get8 ^ 64)));
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const int at = 2048 * FN + 1024 * AL * m;
        if constexpr (XQ) {
          // columns 16 q .. and 64 + 16 q ..: pieces 2 q, 2 q + 1, and those + 8
          const int g = at + 256 * l16, c = 2 * q;
          const uint4 v[4] = {fetch(g + 16 * (c ^ l16)), fetch(g + 16 * ((c + 1) ^ l16)),
                              fetch(g + 16 * ((c + 8) ^ l16)), fetch(g + 16 * ((c + 9) ^ l16))};
          a[m] = quantised_operand(v, e[m]);
        } else {
          a[m] = operand(fetch(at + get8), fetch(at + (get8 ^ 64)));
          e[m] = ev[u][m];
        }
      }
      wave_lds_fence();
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int n = 0; n < FN; ++n)
          add_block<false>(acc[n][m], block_product<false, 0>(b[n], a[m], e[m]), e[m], 0, s[u][n]);
    }
  }
  f32x4* red = reinterpret_cast<f32x4*>(mine) + lane;
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m) red[(n * FM + m) * 64] = acc[n][m];
  __syncthreads();
  for (int t = wave; t < FM * FN; t += W) {
    const uint8_t* at = lds + 1024 * t + 16 * lane;
    f32x4 v = *reinterpret_cast<const f32x4*>(at);
#pragma unroll
    for (int i = 1; i < W; ++i) v += *reinterpret_cast<const f32x4*>(at + i * kWave);
    const int64_t row = m0 + 16 * (t % FM) + l16;
    if (row < p.M) store4<BF16>(p, row, n0 + 16 * (t / FM) + 4 * q, v);
  }
}

template <int FM, int FN, int W, int U, bool XQ, bool BF16>
__global__ __launch_bounds__(64 * W) void linear_rows(LinearArgs p) {
  linear_rows_body<FM, FN, W, U, XQ, BF16>(p);
}

// Larger batches: a workgroup of WM x WN wavefronts computes TM rows x TN
// output features, 128 k (one scale block) per stage. A stage's operands go
// from global memory straight into one of NST LDS buffers (buffer_load ... lds:
// lane l of a wavefront's load fills its 16 bytes at the load's base + 16 l),
// NST - 1 stages ahead of the one that is multiplied.
//   LDS rows are 128 bytes; 16-byte chunk c of row r lies at slot
// c ^ ((r >> 1) & 7), which spreads a fragment read (16 rows, one chunk) over
// all banks. The swizzle is applied on the global side of the load.
//   A wavefront multiplies FN tiles of 16 features with FM tiles of 16 rows.
// The E8M0 bytes of kChunk stages lie in LDS in the order in which a lane
// needs them: byte j of lane l16 is row 16 j + l16, four tiles' bytes to the
// dword, of which the instruction selects one. A wavefront's features lie
// inside one weight block, so one block scale serves its stage.
template <int TM, int TN, int WM, int WN, int NST>
struct LinTile {
  static constexpr int kThreads = 64 * WM * WN;
  static constexpr int FM = TM / WM / 16, FN = TN / WN / 16;
  static constexpr int kStage = (TM + TN) * kLinB;
  static constexpr int LA = TM * 8 / kThreads, LW = TN * 8 / kThreads;  // 16-byte loads a thread
  static constexpr int kLoads = LA + LW;
  static constexpr int kChunk = 32;  // stages whose scales are held
  static constexpr int kBlocks = (TN + kLinB - 1) / kLinB;
  static_assert(TM % (16 * WM) == 0 && TN % (16 * WN) == 0 && kLinB % (TN / WN) == 0, "tiles");
  static_assert(LA * kThreads == TM * 8 && LW * kThreads == TN * 8, "loads");
  static_assert(kThreads / 8 % 16 == 0, "a load's row step keeps the swizzle");
  static_assert(NST >= 2 && NST <= 4 && (NST - 2) * kLoads <= 63, "loads in flight are counted in six bits");
};

// One 16-byte load of each lane into LDS, at lds + 16 lane. It is written as an
// instruction of its own because the compiler, for the builtin, waits for every
// such load in flight before the next LDS read, which would undo the ring; the
// waits are the ring's own (wait_loads). It has no register output. A byte past
// the resource's range is read as zero.
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t voff, u32x4_t rsrc,
                                            uint32_t soff) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
      :
      : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
      : "memory", "m0");
}
__device__ __forceinline__ u32x4_t raw_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4_t{(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, bytes, 0x00020000u};
}
// until at most N of the wavefront's loads are in flight (they end in order)
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0f70);
  asm volatile("" ::: "memory");
}

template <int TM, int TN, int WM, int WN, int NST, bool BF16>
__device__ __forceinline__ void linear_tile_body(const LinearArgs& p, int tiles_m, int tiles_n) {
  using S = LinTile<TM, TN, WM, WN, NST>;
  constexpr int FM = S::FM, FN = S::FN, kChunk = S::kChunk;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[NST * S::kStage];
  __shared__ __attribute__((aligned(16))) uint8_t ex[kChunk * TM];
  __shared__ float sc[S::kBlocks * kChunk];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int tm, tn;
  linear_tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * TM;
  const int n0 = tn * TN;
  const int KB = p.K / kLinB;
  const int mrows = p.M - m0 < TM ? (int)(p.M - m0) : TM;
  const int nrows = p.N - n0 < TN ? p.N - n0 : TN;
  const u32x4_t ar = raw_rsrc(p.codes + m0 * p.K, (uint32_t)mrows * (uint32_t)p.K);
  const u32x4_t wr = raw_rsrc(p.w + (size_t)n0 * p.K, (uint32_t)nrows * (uint32_t)p.K);
  // Load i of this thread takes LDS chunk tid + kThreads i of the operand: a
  // row kThreads / 8 further down each time, which leaves the swizzle alone.
  // Rows past the end lie past the resource's range and read as zero.
  const int r0 = tid >> 3;
  const uint32_t off0 = (uint32_t)r0 * (uint32_t)p.K + 16 * ((tid & 7) ^ ((r0 >> 1) & 7));
  const uint32_t step = (uint32_t)(S::kThreads / 8) * (uint32_t)p.K;
  const uint32_t lds0 =
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)ring + 1024 * wave;
  auto issue = [&](int kb) {
    const uint32_t at = lds0 + (uint32_t)(kb % NST) * S::kStage, k = (uint32_t)(kb * kLinB);
#pragma unroll
    for (int i = 0; i < S::LA; ++i)
      load_to_lds(at + 16 * S::kThreads * i, off0 + i * step, ar, k);
#pragma unroll
    for (int i = 0; i < S::LW; ++i)
      load_to_lds(at + TM * kLinB + 16 * S::kThreads * i, off0 + i * step, wr, k);
  };
  // Scales of the stages kb0 .. kb0 + kChunk - 1. Neighbouring threads read
  // neighbouring bytes of a row's exponents, four at a time if rows are whole,
  // aligned dwords (a byte per row and load, for 128 rows, cost 1.7 us a tile). Row t
  // of the tile is row t % (16 FM) of wavefront row t / (16 FM); what lies past
  // K's end is another row's or 0, and not used.
  const __amdgpu_buffer_rsrc_t er = buffer_rsrc(p.exps + m0 * KB, (uint32_t)mrows * (uint32_t)KB);
  const int nblks = (p.N + kLinB - 1) / kLinB;
  auto scales = [&](int kb0) {
    const auto put = [&](int row, int kb, uint32_t e) {
      ex[kb * TM + (row / (16 * FM)) * (16 * FM) + (row & 15) * FM + (row % (16 * FM)) / 16] =
          (uint8_t)e;
    };
    if (KB % 4 == 0 && reinterpret_cast<uintptr_t>(p.exps) % 4 == 0) {
      constexpr int kPer = kChunk / 4, kN = TM * kPer / S::kThreads;
      static_assert(kN * S::kThreads == TM * kPer, "exponent loads");
      uint32_t e[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int c = tid + S::kThreads * i;
        e[i] = buffer_ld4(er, (uint32_t)(c / kPer) * (uint32_t)KB + kb0 + 4 * (c % kPer));
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int c = tid + S::kThreads * i;
#pragma unroll
        for (int j = 0; j < 4; ++j) put(c / kPer, 4 * (c % kPer) + j, e[i] >> (8 * j));
      }
    } else {
#pragma unroll 4
      for (int c = tid; c < TM * kChunk; c += S::kThreads)
        put(c / kChunk, c % kChunk,
            buffer_ld1(er, (uint32_t)(c / kChunk) * (uint32_t)KB + kb0 + c % kChunk));
    }
    for (int i = tid; i < S::kBlocks * kChunk; i += S::kThreads) {
      const int blk = n0 / kLinB + i / kChunk, kb = kb0 + i % kChunk;
      sc[i] = block_scale<BF16>(
          p.ws[(size_t)(blk < nblks ? blk : nblks - 1) * KB + (kb < KB ? kb : KB - 1)]);
    }
  };

  f32x4 acc[FN][FM];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[n][m] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int sw = (l16 >> 1) & 7;  // fragment rows are multiples of 16 plus l16
  const int abyte = (wm * 16 * FM + l16) * kLinB;
  const int wbyte = TM * kLinB + (wn * 16 * FN + l16) * kLinB;
  const int c0 = 16 * (q ^ sw), c1 = 16 * ((q + 4) ^ sw);
  auto fragment = [&](const uint8_t* row) {
    return operand(*reinterpret_cast<const uint4*>(row + c0),
                   *reinterpret_cast<const uint4*>(row + c1));
  };
  auto compute = [&](int kb) {
    const uint8_t* buf = ring + (kb % NST) * S::kStage;
    const uint8_t* e = ex + (kb % kChunk) * TM + wm * 16 * FM + l16 * FM;
    const float s = sc[(wn * 16 * FN / kLinB) * kChunk + kb % kChunk];
    uint32_t ew[(FM + 3) / 4];
    if constexpr (FM >= 4) {
#pragma unroll
      for (int j = 0; j < FM / 4; ++j) ew[j] = *reinterpret_cast<const uint32_t*>(e + 4 * j);
    } else {
      ew[0] = 0;
#pragma unroll
      for (int j = 0; j < FM; ++j) ew[0] |= (uint32_t)e[j] << (8 * j);
    }
    i32x8_t w[FN];
#pragma unroll
    for (int n = 0; n < FN; ++n) w[n] = fragment(buf + wbyte + n * 16 * kLinB);
    // Row tile m's products start as tile m - 1's are scaled and added: the
    // additions of d[n] stand before the product that overwrites it, FN
    // products after the one they wait for. The barriers and pin() keep the
    // compiler to this order (it would add a product right after its start,
    // and gather fragments it has no registers for).
    i32x8_t a = fragment(buf + abyte);
    f32x4 d[FN];
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      i32x8_t next = a;
      if (m + 1 < FM) next = fragment(buf + abyte + (m + 1) * 16 * kLinB);
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        if (m > 0) {
          pin(d[n]);
          add_block<BF16>(acc[n][m - 1], d[n], (int)ew[(m - 1) / 4], (m - 1) & 3, s);
        }
        d[n] = block_product_sel<BF16>(w[n], a, (int)ew[m / 4], m & 3);
        __builtin_amdgcn_sched_barrier(0);
      }
      a = next;
    }
#pragma unroll
    for (int n = 0; n < FN; ++n)
      add_block<BF16>(acc[n][FM - 1], d[n], (int)ew[(FM - 1) / 4], (FM - 1) & 3, s);
  };
#pragma unroll
  for (int i = 0; i < NST - 1; ++i)
    if (i < KB) issue(i);
#pragma unroll 1
  for (int kb = 0; kb < KB; ++kb) {
    if (kb % kChunk == 0) {
      if (kb > 0) lds_barrier();  // the last chunk's scales have been read
      scales(kb);
    }
    // this stage's loads have ended once only those of the stages after it,
    // NST - 2 at most, are in flight
    const int later = KB - 1 - kb < NST - 2 ? KB - 1 - kb : NST - 2;
    if (later <= 0)
      wait_loads<0>();
    else if (later == 1)
      wait_loads<S::kLoads>();
    else
      wait_loads<2 * S::kLoads>();
    // every wavefront's part is there, and the buffer read last is free
    lds_barrier();
    if (kb + NST - 1 < KB) issue(kb + NST - 1);
    compute(kb);
  }
  // bf16 rows of whole 16-byte pieces go out through LDS (the ring is free):
  // a lane's four features of a row are half a piece, and lines of the output
  // written in one go spare the memory system the merging (8192 x 8192 x 4096:
  // 253 to 240 us).
  if constexpr (BF16 && 16 * FN * 2 == 128) {
    if (p.vec8 && n0 + TN <= p.N) {
      static_assert(FM * 16 * 128 * WM * WN <= NST * S::kStage, "the output tile fits the ring");
      lds_barrier();
      uint8_t* mine = ring + wave * (FM * 16 * 128);
      const int col = n0 + wn * 16 * FN;
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        f32x4 b = {0.f, 0.f, 0.f, 0.f};
        if (p.bias) {
#pragma unroll
          for (int j = 0; j < 4; ++j) b[j] = p.bias[col + 16 * n + 4 * q + j];
        }
#pragma unroll
        for (int m = 0; m < FM; ++m) {
          const f32x4 v = acc[n][m] + b;
          const int piece = (2 * n + (q >> 1)) ^ (l16 & 7);
          *reinterpret_cast<uint2*>(mine + (16 * m + l16) * 128 + 16 * piece + 8 * (q & 1)) =
              make_uint2(f32_to_bf16_bits(v[0]) | f32_to_bf16_bits(v[1]) << 16,
                         f32_to_bf16_bits(v[2]) | f32_to_bf16_bits(v[3]) << 16);
        }
      }
      const int64_t row0 = m0 + wm * 16 * FM;
      uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + row0 * p.ld_out + col;
#pragma unroll
      for (int i = 0; i < 2 * FM; ++i) {
        const int r = 8 * i + (lane >> 3), c = lane & 7;
        const uint4 v = *reinterpret_cast<const uint4*>(mine + r * 128 + 16 * (c ^ (r & 7)));
        if (row0 + r < p.M) *reinterpret_cast<uint4*>(out + (int64_t)r * p.ld_out + 8 * c) = v;
      }
      return;
    }
  }
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int64_t row = m0 + wm * 16 * FM + 16 * m + l16;
    if (row >= p.M) continue;
#pragma unroll
    for (int n = 0; n < FN; ++n)
      store4<BF16>(p, row, n0 + wn * 16 * FN + 16 * n + 4 * q, acc[n][m]);
  }
}

template <int TM, int TN, int WM, int WN, int NST, bool BF16>
__global__ __launch_bounds__(64 * WM * WN) void linear_tile(LinearArgs p, int tiles_m,
                                                           int tiles_n) {
  linear_tile_body<TM, TN, WM, WN, NST, BF16>(p, tiles_m, tiles_n);
}

static size_t al256(size_t n) { return (n + 255) / 256 * 256; }

template <int TM, int TN, int WM, int WN, int NST, bool BF16>
static void launch_tile(const LinearArgs& p, hipStream_t s) {
  const int tm = (int)((p.M + TM - 1) / TM), tn = (p.N + TN - 1) / TN;
  linear_tile<TM, TN, WM, WN, NST, BF16><<<(unsigned)((int64_t)tm * tn), 64 * WM * WN, 0, s>>>(p, tm, tn);
}

template <int FM, int FN, int W, int U, bool XQ, bool BF16>
static void launch_rows(const LinearArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.N + 16 * FN - 1) / (16 * FN)),
                  (unsigned)((p.M + 16 * FM - 1) / (16 * FM)));
  linear_rows<FM, FN, W, U, XQ, BF16><<<grid, 64 * W, 0, s>>>(p);
}

constexpr int kUnits = 256;  // compute units
static int64_t tiles_of(int64_t M, int N, int tm, int tn) {
  return (M + tm - 1) / tm * ((N + tn - 1) / tn);
}

// Whether the product quantises bf16 rows itself. Its workgroups then read x at
// two bytes and each repeat the conversion for their own features: K = 1024 +
// 1.1 us, 2048 + 2.0, 4096 + 3.7 (77 x 2112), where a launch of the quantiser
// takes 3.1 and the gap to the next one 1 (measured up to 128 rows).
static bool quantises_inside(int64_t M, int N, int K) {
  return M <= 16 || (M <= 128 && K <= 32 * kLinB && tiles_of(M, N, 32, 32) <= kUnits);
}

// Which kernel a product runs on. Times in us on one MI355X for K = 4096 (they
// go with K), weights not in any cache.
//
// Up to 16 rows: the stream, 16 features a workgroup, or 32 where that would
// ask for a second round of them (16 x 8192: 32 features 9.4, 16 features 13.2;
// 16 x 4096: 8.3 and 7.4). A wavefront requests two blocks at a time if K has
// them (16 x 4096: 7.4, one at a time 8.8; at K = 2048, where every second
// would be for nothing, 5.6 and 4.5).
//
// Above, while one round of workgroups, one a compute unit, covers the product:
// the stream with the fewest rows and features a workgroup that does so, since
// a compute unit's time goes with what it reads: 32 x 16 7.1 (24 x 4096), 32 x
// 32 8.2, 48 x 32 10.0, 64 x 32 11.9, 48 x 64 12.7, 64 x 64 14.7; the smallest
// tile 15.4.
//
// Tiles: the kind whose rounds of workgroups cost least. A round, with as many
// workgroups as fit the chip at once:
//   bf16 output   256 x 256   256 workgroups  62     128 x 256   256  39
//                 128 x 128   512 (two a compute unit)  41, or 256 with a
//                             deeper ring  26          64 x 64    512  20
//   fp32 output   128 x 256   256  69     128 x 128   256  41     64 x 64   512  29
// (bf16: 2048 x 4096: 56 / 39 / 41 / 49 / 63; 1000 x 4096: 54 / 34 / 32 / 26 /
// 38; 500 x 4096: 64 x 64 21; 8192 x 8192: 240 / 283 / 292 / 367 / 432. fp32:
// 2048 x 4096: 69 / 82 / 88; 1000 x 4096: 66 / 44 / 50; 300 x 4096: 128 x 128
// 41, 64 x 64 28; 8192 x 8192: 535 / 642 / 707.)
template <int FN, bool XQ, bool BF16>
static void launch_16(const LinearArgs& p, hipStream_t s) {
  if (p.K > 16 * kLinB)
    launch_rows<1, FN, 16, 2, XQ, BF16>(p, s);
  else
    launch_rows<1, FN, 16, 1, XQ, BF16>(p, s);
}

template <bool BF16>
static void launch_form(const LinearArgs& p, hipStream_t s) {
  const auto blocks = [&](int tm, int tn) { return tiles_of(p.M, p.N, tm, tn); };
  if (p.M <= 16) {
    if (blocks(16, 16) > kUnits)
      return p.x ? launch_16<2, true, BF16>(p, s) : launch_16<2, false, BF16>(p, s);
    return p.x ? launch_16<1, true, BF16>(p, s) : launch_16<1, false, BF16>(p, s);
  }
  if (blocks(32, 16) <= kUnits)
    return p.x               ? launch_rows<2, 1, 16, 1, true, BF16>(p, s)
           : p.K > 16 * kLinB ? launch_rows<2, 1, 16, 2, false, BF16>(p, s)
                              : launch_rows<2, 1, 16, 1, false, BF16>(p, s);
  if (blocks(32, 32) <= kUnits)
    return p.x ? launch_rows<2, 2, 8, 1, true, BF16>(p, s)
               : launch_rows<2, 2, 8, 1, false, BF16>(p, s);
  if (blocks(48, 32) <= kUnits) return launch_rows<3, 2, 8, 1, false, BF16>(p, s);
  if (blocks(64, 32) <= kUnits) return launch_rows<4, 2, 8, 1, false, BF16>(p, s);
  if (blocks(48, 64) <= kUnits) return launch_rows<3, 4, 8, 1, false, BF16>(p, s);
  if (blocks(64, 64) <= kUnits) return launch_rows<4, 4, 8, 1, false, BF16>(p, s);
  const auto cost = [&](int tm, int tn, int round, int us) {
    return (blocks(tm, tn) + round - 1) / round * us;
  };
  if constexpr (BF16) {
    const int64_t t[] = {cost(64, 64, 512, 20), cost(128, 128, 256, 26), cost(128, 128, 512, 41),
                         cost(128, 256, 256, 39), cost(256, 256, 256, 62)};
    int best = 0;
    for (int i = 1; i < 5; ++i)
      if (t[i] < t[best]) best = i;
    switch (best) {
      case 0: return launch_tile<64, 64, 4, 1, 3, BF16>(p, s);
      case 1: return launch_tile<128, 128, 4, 2, 4, BF16>(p, s);
      case 2: return launch_tile<128, 128, 4, 2, 2, BF16>(p, s);
      case 3: return launch_tile<128, 256, 2, 4, 3, BF16>(p, s);
      default: return launch_tile<256, 256, 2, 4, 2, BF16>(p, s);
    }
  } else {
    const int64_t t0 = cost(64, 64, 512, 29), t1 = cost(128, 128, 256, 41),
                  t2 = cost(128, 256, 256, 69);
    if (t0 <= t1 && t0 <= t2) return launch_tile<64, 64, 2, 2, 2, BF16>(p, s);
    if (t1 <= t2) return launch_tile<128, 128, 4, 2, 2, BF16>(p, s);
    launch_tile<128, 256, 2, 4, 3, BF16>(p, s);
  }
}

static hipError_t launch_linear(const LinearArgs& p, bool bf16, hipStream_t s) {
  if (bf16)
    launch_form<true>(p, s);
  else
    launch_form<false>(p, s);
  return hipGetLastError();
}

static moe_status check_sizes(int64_t M, int32_t N, int32_t K) {
  if (M < 0 || N <= 0 || K <= 0) return MOE_ERR_SHAPE;
  if (K % kLinB != 0) return MOE_ERR_UNSUPPORTED;
  // 32-bit offsets within a tile, fewer than 2^32 threads a grid (at most one
  // for 64 outputs where there are many), and the quantiser's grid
  if (K > (1 << 22) || N > (1 << 24) || M > (1 << 20) ||
      (M + 15) / 16 * ((N + 63) / 64) >= ((int64_t)1 << 27) ||
      M * (K / kLinB) >= ((int64_t)1 << 27))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

static moe_status linear_call(LinearArgs p, moe_dtype out_dtype, void* workspace,
                              size_t workspace_bytes, hipStream_t s) {
  const moe_status st = check_sizes(p.M, p.N, p.K);
  if (st != MOE_OK) return st;
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16) return MOE_ERR_SHAPE;
  if (p.ld_out < p.N || (p.x && p.ld_x < p.K)) return MOE_ERR_SHAPE;
  if (p.M == 0) return MOE_OK;
  const auto odd16 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 != 0; };
  if (odd16(p.x) || odd16(p.codes) || odd16(p.w) || (p.x && p.ld_x % 8 != 0))
    return MOE_ERR_UNSUPPORTED;
  const size_t need = moe_linear_workspace_bytes(p.M, p.N, p.K, p.x ? 0 : 1);
  if (need > 0) {
    if (!workspace) return MOE_ERR_NULL;
    if (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
      return MOE_ERR_WORKSPACE;
  }
  if (p.x && !quantises_inside(p.M, p.N, p.K)) {
    uint8_t* codes = static_cast<uint8_t*>(workspace);
    uint8_t* exps = codes + al256((size_t)p.M * p.K);
    if (launch_quant_act(p.x, p.M, p.K, codes, exps, s, p.ld_x) != hipSuccess) return MOE_ERR_HIP;
    p.x = nullptr;
    p.codes = codes;
    p.exps = exps;
  }
  const size_t quad = out_dtype == MOE_BF16 ? 8 : 16;
  p.vec4 = reinterpret_cast<uintptr_t>(p.out) % quad == 0 && p.ld_out % 4 == 0;
  p.vec8 = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.ld_out % 8 == 0;
  return launch_linear(p, out_dtype == MOE_BF16, s) == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_linear_workspace_bytes(int64_t rows, int32_t out_features, int32_t in_features,
                                  int32_t x_is_codes) {
  if (check_sizes(rows, out_features, in_features) != MOE_OK || rows == 0) return 0;
  if (x_is_codes || quantises_inside(rows, out_features, in_features)) return 0;
  return al256((size_t)rows * in_features) + al256((size_t)rows * (in_features / kLinB));
}

moe_status moe_linear(const void* x, int64_t ld_x, const uint8_t* w, const float* w_scales,
                      const float* bias, int64_t rows, int32_t out_features, int32_t in_features,
                      void* out, int64_t ld_out, moe_dtype out_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!x || !w || !w_scales || !out) return MOE_ERR_NULL;
  LinearArgs p{};
  p.x = static_cast<const uint16_t*>(x);
  p.ld_x = ld_x;
  p.w = w;
  p.ws = w_scales;
  p.bias = bias;
  p.out = out;
  p.M = rows;
  p.ld_out = ld_out;
  p.N = out_features;
  p.K = in_features;
  return linear_call(p, out_dtype, workspace, workspace_bytes, static_cast<hipStream_t>(stream));
}

moe_status moe_linear_e4m3(const uint8_t* codes, const uint8_t* exps, const uint8_t* w,
                           const float* w_scales, const float* bias, int64_t rows,
                           int32_t out_features, int32_t in_features, void* out, int64_t ld_out,
                           moe_dtype out_dtype, void* workspace, size_t workspace_bytes,
                           void* stream) {
  if (!codes || !exps || !w || !w_scales || !out) return MOE_ERR_NULL;
  LinearArgs p{};
  p.codes = codes;
  p.exps = exps;
  p.w = w;
  p.ws = w_scales;
  p.bias = bias;
  p.out = out;
  p.M = rows;
  p.ld_out = ld_out;
  p.N = out_features;
  p.K = in_features;
  return linear_call(p, out_dtype, workspace, workspace_bytes, static_cast<hipStream_t>(stream));
}

}  // extern "C"
