// linear_w4.hpp — the kernels of moe_linear_w4 and moe_grouped_linear_w4: products
// with 4-bit weights,
//   out[t][n] = sum_k x[t][k] (q[n][k] - z[n][g]) s[n][g] (+ bias[n]),  g = k / G,
// one bank for all rows, or one bank an expert for rows sorted by expert.
//
// A group's sum is split as s (sum_k x q - z sum_k x): the matrix instruction
// multiplies bf16 rows of x with the codes themselves, which bf16 holds exactly,
// and fp32 takes scale and zero point. Nothing is rounded before the output.
// The codes get to bf16 as E4M3 bytes: byte q (0 .. 15) is the E4M3 number q 2^-9
// (0 .. 7 are its subnormals, 8 .. 15 its first binade), so a masked nibble is
// already an operand of the conversion instruction. The factor 2^9 goes into s.
#pragma once

#include "device.hpp"
#include "layer.hpp"

#include <type_traits>

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

// The tiles of at most TM rows of all experts, one expert after the other: lane l
// counts those of experts [C l, C (l + 1)), a scan gives the tiles before them, and
// the lane whose tiles hold a slot tells the others. All offsets are requested at
// once: one after the other they took 5 us of a decode batch's call on 512 experts.
// Offsets are cut to [0, M].
template <int TM, int C>
struct Tiles {
  int at[C + 1], before, tiles, total;
  __device__ __forceinline__ void read(const W4Args& p) {
    const int e0 = (int)(threadIdx.x & 63) * C, M = (int)p.M;
#pragma unroll
    for (int i = 0; i <= C; ++i) at[i] = p.offsets[e0 + i < p.E ? e0 + i : p.E];
    tiles = 0;
#pragma unroll
    for (int i = 0; i <= C; ++i) at[i] = at[i] < 0 ? 0 : at[i] > M ? M : at[i];
#pragma unroll
    for (int i = 0; i < C; ++i) tiles += count(i);
    const int incl = wave_incl_scan(tiles);
    before = incl - tiles;
    total = __builtin_amdgcn_readlane(incl, 63);
  }
  __device__ __forceinline__ int count(int i) const {
    return at[i + 1] > at[i] ? (at[i + 1] - at[i] + TM - 1) / TM : 0;
  }
  __device__ __forceinline__ RowTile find(int slot) const {
    int left = slot - before, e = 0, r0 = 0, rows = 0;
    const uint64_t owners = __ballot(left >= 0 && left < tiles);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int n = count(i);
      if (left >= 0 && left < n) {
        e = (int)(threadIdx.x & 63) * C + i;
        r0 = at[i] + left * TM;
        rows = at[i + 1] - r0 < TM ? at[i + 1] - r0 : TM;
      }
      left -= n;
    }
    RowTile r{0, 0, 0};
    if (owners == 0) return r;
    const int owner = __builtin_ctzll(owners);
    r.e = __builtin_amdgcn_readlane(e, owner);
    r.rows = __builtin_amdgcn_readlane(rows, owner);
    r.r0 = __builtin_amdgcn_readlane(r0, owner);
    return r;
  }
};
template <int TM, int C>
__device__ __forceinline__ RowTile find_grouped(const W4Args& p, int slot) {
  Tiles<TM, C> t;
  t.read(p);
  return t.find(slot);
}
template <int TM>
__device__ __forceinline__ RowTile dense_tile(const W4Args& p, int slot) {
  const int64_t r0 = (int64_t)slot * TM, left = p.M - r0;
  return RowTile{0, left < TM ? (int)left : TM, r0};
}
template <int TM>
__device__ __forceinline__ RowTile find_tile(const W4Args& p, int slot) {
  if (!p.offsets) return dense_tile<TM>(p, slot);
  if (p.E <= 128) return find_grouped<TM, 2>(p, slot);
  if (p.E <= 512) return find_grouped<TM, 8>(p, slot);
  return find_grouped<TM, 16>(p, slot);
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

constexpr int kW4Units = 256;  // compute units
constexpr float kCodeScale = 512.f;  // 2^9: a code's operand is q 2^-9

__device__ __forceinline__ float w4_silu(float g) { return g / (1.f + expf(-g)); }
__device__ __forceinline__ void w4_store(const W4Args& p, int64_t row, int n, float v) {
  if (p.out_bf16)
    static_cast<__bf16*>(p.out)[row * p.ld_out + n] = (__bf16)v;
  else
    static_cast<float*>(p.out)[row * p.ld_out + n] = v;
}

// Loads straight into LDS: lane l's piece (16 bytes; or one value, widened to a
// dword) goes to lds + 16 l (4 l). Instructions of their own: for the builtin the
// compiler waits for every such load before the next LDS read. They have no register
// output; what reads the piece waits first (w4_wait).
__device__ __forceinline__ const void* uniform(const void* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const void*>(
      (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a) |
      (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) << 32);
}
__device__ __forceinline__ void lds16(uint32_t lds, const void* base, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(uniform(base))
               : "memory", "m0");
}
template <int BYTES>
__device__ __forceinline__ void lds4(uint32_t lds, const void* base, uint32_t off) {
  if (BYTES == 4)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "memory", "m0");
  else if (BYTES == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ushort %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, %2"
                 :
                 : "s"(lds), "v"(off), "s"(base)
                 : "memory", "m0");
}
// The same with 64-bit addresses.
template <int BYTES>
__device__ __forceinline__ void lds4_at(uint32_t lds, const void* at) {
  const uint32_t to = __builtin_amdgcn_readfirstlane(lds);
  if (BYTES == 4)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
                 :
                 : "s"(to), "v"(at)
                 : "memory", "m0");
  else if (BYTES == 2)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ushort %1, off"
                 :
                 : "s"(to), "v"(at)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, off"
                 :
                 : "s"(to), "v"(at)
                 : "memory", "m0");
}
// until at most N of the wavefront's vector memory operations are under way (loads
// end in order), and none of its LDS reads
template <int N>
__device__ __forceinline__ void w4_wait() {
  static_assert(N >= 0 && N <= 63, "six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0070);
  asm volatile("" ::: "memory");
}
template <class T>
__device__ __forceinline__ uint32_t lds_offset(T* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) T*)p;
}

// Few rows: a stream of the weights. All strips of 16 weight rows of all tiles of
// 16 rows are shared out evenly among the workgroups, so that each takes runs of
// strips of one tile, or two. A workgroup's W wavefronts share K, UW units of 128
// columns each, whose x they hold in registers for a run (if K is longer than W UW
// units, in several passes a strip, x read again). A strip's codes, scales and zero
// points go straight to LDS, D - 1 strips ahead of the one that is multiplied: what
// bounds the stream is the bytes under way (one strip ahead, in registers, 8
// wavefronts a compute unit: 15 B/ns a unit, 3.9 TB/s). A wavefront reads nothing
// but its own pieces, so that the ring needs no barrier. The partial sums meet in
// LDS, two buffers in turn, and are added in wavefront order.
//   Lane l reads 16 bytes (32 codes) of weight row l % 16 at quarter l / 16 of the
// unit; after the exchange between the quarters instruction b covers the unit's
// columns 32 b .. 32 b + 31, so that every group size is a whole number of
// instructions. x is the A operand: a lane ends with four rows of one output
// feature, whose scale it holds itself. The sums of x over the groups come from the
// same instruction, with ones (2^-9) for the weights. With swiglu a strip of gates
// and the strip of their ups follow each other; the thread that adds a gate's
// partial sums keeps it for its up's.
//   Measured: one layer's banks of a decode batch, 197 MB in two calls, 48 to 52 us (4
// TB/s); 321 MB of one bank 64 us (5.0 TB/s). 128 rows of 4096 x 4096: 18 us, of
// which vector instructions (exchange, conversions, scales) fill 8 and matrix instructions
// 2; two wavefronts a SIMD wait for the rest (22 with x read again from the L2 for each
// strip).
template <int G, bool Z, int W, int UW, int KB>
struct StreamRing {
  static constexpr int kGroups = UW * 128 / G;          // a wavefront's groups in a row
  static constexpr int kScaleLoads = (kGroups + 3) / 4;  // 16 rows x 4 groups each
  static constexpr int kLoads = UW + kScaleLoads * (Z ? 2 : 1) + 1;
  static constexpr int kScales = UW * 1024, kZeros = kScales + 256 * kScaleLoads,
                       kBias = kZeros + (Z ? 256 * kScaleLoads : 0), kSlot = kBias + 256;
  // strips in the ring: what KB KiB hold beside the partial sums
  static constexpr int kFit = (KB * 1024 - 2 * W * 1024 - 64) / (W * kSlot);
  static constexpr int kCount = 2 + 63 / kLoads;  // (waits count six bits)
  static constexpr int D = kFit < kCount ? kFit : kCount;
  static_assert(D >= 2 && (D - 2) * kLoads <= 63, "the ring");
  static constexpr int kBytes = W * D * kSlot;
};
template <int G, bool SB, bool Z, int W, int UW, int KB, bool LONG>
__global__ __launch_bounds__(64 * W, 2) void w4_stream(W4Args p) {
  using R = StreamRing<G, Z, W, UW, KB>;
  constexpr int D = R::D;
  constexpr int TM = 16, NG = 128 / G, NB = G / 32, kOut = (TM * 16 + 64 * W - 1) / (64 * W);
  __shared__ __attribute__((aligned(16))) uint8_t ring[R::kBytes];
  __shared__ float part[2][W][4][64];
  __shared__ __attribute__((aligned(16))) int32_t plan[4];  // tiles; the tile in hand
  const int tid = threadIdx.x, lane = tid & 63, l = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n_out = p.swiglu ? p.N / 2 : p.N, strips = (n_out + 15) / 16, groups = p.K / G;
  const int per = p.swiglu ? 2 : 1;
  const int passes = LONG ? (p.K + 128 * W * UW - 1) / (128 * W * UW) : 1;
  uint8_t* const mine = ring + w * (D * R::kSlot);
  const uint32_t lds0 = lds_offset(mine);
  // This workgroup's share of all strips of all tiles, and the tile of its first one
  // (slot < 0) or the slot-th. Wavefront 0 looks it up for all.
  int cur, end;
  const auto share = [&](int tiles) {
    // (offsets that do not ascend could count rows twice: no more tiles than rows and
    // experts allow; of the sizes that take the stream they are below 2^29 strips)
    const int most = (int)p.M / TM + (int)(p.M < p.E ? p.M : p.E);
    const uint64_t all = (uint64_t)(p.offsets && tiles > most ? most : tiles) * (uint64_t)strips;
    cur = __builtin_amdgcn_readfirstlane((int)(all * blockIdx.x / gridDim.x));
    end = __builtin_amdgcn_readfirstlane((int)(all * (blockIdx.x + 1) / gridDim.x));
  };
  const auto look_up = [&](auto t, int slot) {
    t.read(p);
    if (slot < 0) {
      share(t.total);
      slot = cur / strips;
    }
    const RowTile r = t.find(slot);
    if (lane == 0) *reinterpret_cast<int4*>(plan) = make_int4(t.total, r.e, r.rows, (int)r.r0);
  };
  RowTile tile;
  const auto locate = [&](int slot) {
    if (!p.offsets) {
      if (slot < 0) {
        share((int)((p.M + TM - 1) / TM));
        slot = cur / strips;
      }
      tile = dense_tile<TM>(p, slot);
      return;
    }
    lds_barrier();  // (the last tile's plan has been read)
    if (w == 0) {
      if (p.E <= 128)
        look_up(Tiles<TM, 2>{}, slot);
      else if (p.E <= 512)
        look_up(Tiles<TM, 8>{}, slot);
      else
        look_up(Tiles<TM, 16>{}, slot);
    }
    lds_barrier();
    if (slot < 0) share(__builtin_amdgcn_readfirstlane(plan[0]));
    tile.e = __builtin_amdgcn_readfirstlane(plan[1]);
    tile.rows = __builtin_amdgcn_readfirstlane(plan[2]);
    tile.r0 = __builtin_amdgcn_readfirstlane(plan[3]);
  };
  // (the sum that starts a product without zero points is -8 times that of x)
  const float one = !Z && G == 32 ? -8.f / kCodeScale : 1.f / kCodeScale;
  bf16x8_t ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = (__bf16)one;
  // where the stream is: strip, its half (gates, ups) and its pass over K
  struct At {
    int strip, half, pass;
  };
  const auto step = [&](At& at) {
    if (++at.pass < passes) return;
    at.pass = 0;
    if (++at.half < per) return;
    at.half = 0;
    ++at.strip;
  };
  const auto unit = [&](int pass, int u) { return 128 * ((pass * W + w) * UW + u); };
  int buffer = 0;  // of the ring, of the strip that is multiplied next
  int sums = 0;    // of the partial sums: in turn over all runs, as nothing else parts them
  locate(-1);
#pragma unroll 1
  while (cur < end) {
    const int s0 = cur % strips, s1 = end - cur < strips - s0 ? s0 + end - cur : strips;
    cur += s1 - s0;
    const int64_t bank = (int64_t)tile.e * p.N;
    // one strip's pieces into ring buffer b; rows past the last repeat it, and so do
    // columns behind K, for which x counts as zero: any code will do
    const auto issue = [&](const At& at, int b) {
      const uint32_t to = __builtin_amdgcn_readfirstlane(lds0 + b * R::kSlot);
      const int left = n_out - 16 * at.strip;
      const int64_t n = bank + 16 * at.strip + at.half * n_out;
      const auto row = [&](int r) { return r < left ? r : left - 1; };
      const uint8_t* wp = p.w + n * (p.K / 2);
#pragma unroll
      for (int u = 0; u < UW; ++u) {
        const int k = unit(at.pass, u) + 32 * q;
        lds16(to + 1024 * u, wp, (uint32_t)(row(l) * (p.K / 2) + (k < p.K ? k : 0) / 2));
      }
      const uint8_t* sp = static_cast<const uint8_t*>(p.ws) + n * groups * (SB ? 2 : 4);
#pragma unroll
      for (int i = 0; i < R::kScaleLoads; ++i) {  // lane: row lane / 4, group lane % 4
        const int k = unit(at.pass, 0) / G + 4 * i + (lane & 3);
        const uint32_t o = (uint32_t)(row(lane >> 2) * groups + (k < groups ? k : groups - 1));
        lds4<SB ? 2 : 4>(to + R::kScales + 256 * i, sp, o * (SB ? 2 : 4));
        if (Z) lds4<1>(to + R::kZeros + 256 * i, p.wz + n * groups, o);
      }
      // (without a bias the value is not used: w has four bytes a feature, too)
      const float* bp = p.bias ? p.bias : reinterpret_cast<const float*>(p.w);
      lds4<4>(to + R::kBias, bp + n, 4u * (uint32_t)row(l));
    };
    const uint16_t* xp = p.x + (tile.r0 + (l < tile.rows ? l : tile.rows - 1)) * p.ld_x;
    // x in the codes' order, and the groups' sums (without zero points: times -8, what
    // a group's product starts from)
    // (groups of 32 columns: 64 registers; there the instruction is repeated instead)
    constexpr bool kHeld = G > 32;
    bf16x8_t a[UW][4];
    f32x4 xs[kHeld ? UW : 1][NG];
    const auto load_x = [&](int pass) {
#pragma unroll
      for (int u0 = 0; u0 < UW; u0 += 2) {  // (two units under way: registers)
        uint4 v[2][4];
#pragma unroll
        for (int u = u0; u < u0 + 2 && u < UW; ++u)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int k = unit(pass, u) + 32 * b;
            v[u - u0][b] = make_uint4(0, 0, 0, 0);
            if (k < p.K) v[u - u0][b] = ld16(xp + k + 8 * q);
          }
#pragma unroll
        for (int u = u0; u < u0 + 2 && u < UW; ++u)
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = g * NB; b < (g + 1) * NB; ++b) {
              a[u][b] = x_order(v[u - u0][b]);
              if (kHeld) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[u][b], ones, sum, 0, 0, 0);
            }
            if (kHeld) {
#pragma unroll
              for (int j = 0; j < 4; ++j) xs[u][g][j] = Z ? sum[j] : -8.f * sum[j];
            }
          }
      }
    };
    At at{s0, 0, 0}, ahead = at;
    int issued = 0, done = 0;
    const int items = (s1 - s0) * per * passes;
#pragma unroll 1
    for (; issued < D - 1 && issued < items; ++issued) {
      issue(ahead, (buffer + issued) % D);
      step(ahead);
    }
    load_x(0);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    float gate[kOut];
#pragma unroll 1
    for (; done < items; ++done) {
      if (LONG && done > 0) load_x(at.pass);
      if (issued - done - 1 >= D - 2)
        w4_wait<(D - 2) * R::kLoads>();
      else
        w4_wait<0>();
      const uint8_t* from = mine + buffer * R::kSlot;
      uint4 code[UW];
#pragma unroll
      for (int u = 0; u < UW; ++u) code[u] = *reinterpret_cast<const uint4*>(from + 1024 * u + 16 * lane);
      const float bias = *reinterpret_cast<const float*>(from + R::kBias + 4 * l);
      // (the buffer before this one has been read: w4_wait)
      if (issued < items) {
        issue(ahead, buffer == 0 ? D - 1 : buffer - 1);
        step(ahead);
        ++issued;
      }
      buffer = buffer + 1 == D ? 0 : buffer + 1;
      uint32_t s4[4], z4[4];  // raw scales and zero points of four groups
#pragma unroll
      for (int u = 0; u < UW; ++u) {
        transpose_quarters(code[u]);
        const uint32_t cw[4] = {code[u].x, code[u].y, code[u].z, code[u].w};
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int at4 = u * NG + g;
          if (at4 % 4 == 0) {
            const uint4 sv = *reinterpret_cast<const uint4*>(from + R::kScales + 64 * at4 + 16 * l);
            s4[0] = sv.x, s4[1] = sv.y, s4[2] = sv.z, s4[3] = sv.w;
            if (Z) {
              const uint4 zv = *reinterpret_cast<const uint4*>(from + R::kZeros + 64 * at4 + 16 * l);
              z4[0] = zv.x, z4[1] = zv.y, z4[2] = zv.z, z4[3] = zv.w;
            }
          }
          f32x4 xg;
          if (kHeld) {
            xg = xs[kHeld ? u : 0][g];
          } else {
            asm volatile("" : "+v"(ones));  // (or it is done ahead, and held)
            xg = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[u][g], ones, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
          }
          f32x4 d = Z ? f32x4{0.f, 0.f, 0.f, 0.f} : xg;
#pragma unroll
          for (int b = g * NB; b < (g + 1) * NB; ++b)
            d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[u][b], codes_bf16(cw[b]), d, 0, 0, 0);
          const float sv = __uint_as_float(s4[at4 % 4] << (SB ? 16 : 0));
          const float zv = Z ? -(float)z4[at4 % 4] : 0.f;
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[v] = fmaf(sv, Z ? fmaf(zv, xg[v], d[v]) : d[v], acc[v]);
        }
      }
      if (at.pass + 1 == passes) {
        float (*buf)[4][64] = part[sums];
        sums ^= 1;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          buf[w][v][lane] = acc[v];
          acc[v] = 0.f;
        }
        lds_barrier();  // (a buffer is written again only behind the next strip's barrier)
        // value (row r, feature c) lies at lane 16 (r / 4) + c, v = r % 4
#pragma unroll
        for (int o = 0; o < kOut; ++o) {
          const int i = tid + 64 * W * o, r = i / 16, n = 16 * at.strip + l;
          if (r >= tile.rows || n >= n_out) continue;
          float y = 0.f;
#pragma unroll
          for (int ww = 0; ww < W; ++ww) y += buf[ww][r & 3][16 * (r >> 2) + l];
          y *= kCodeScale;
          if (p.bias) y += bias;
          if (per == 2) {
            if (at.half == 0) {
              gate[o] = y;
              continue;
            }
            y = w4_silu(gate[o]) * y;
          }
          w4_store(p, tile.r0 + r, n, y);
        }
      }
      step(at);
    }
    if (cur < end) locate(cur / strips);
  }
}

// ------------------------------------------------------------ larger batches --
// bf16 output of larger batches: both operands become fp16, so that scale and
// zero point are in the weight itself and the matrix instructions run one chain of
// sums over all of K.
//   x: bf16 has 8 significant bits and fp16 11, so a row times a power of two that
// brings its largest magnitude into [2^14, 2^15) is exact down to 2^-29 of that
// magnitude (and off by at most 2^-25, 2^-39 of it, below). w4_halves writes such rows to the
// workspace, with columns in the order in which codes leave a dword.
//   W: a masked code is the fp16 subnormal q 2^-24 (16 q 2^-24 for the upper four
// bits of a byte), so one multiply-add with 2^15 (2^11) and -z 2^-9 makes it
// (q - z) 2^-9, exact, and one multiplication with S the weight: 13 instructions for
// eight. S is s times the power of two of the weights' row that brings its largest
// into [2^14, 2^15). S and the product are rounded to fp16's 11 bits, which moves a
// weight by at most 2^-10 of itself (S of a bf16 scale is exact: by 2^-11), and by
// 2^-29 of the row's largest scale where it is below fp16's normal numbers.
// (z s is never rounded apart from q s: what that leaves is common to a group's
// columns, and adds up over rows that have a mean. The exact form takes a multiply-add
// on each sum and group besides.)
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kW4Stage = 128;  // columns of a stage

// Rows of x as fp16 x 2^-e [M][Kp], zeros behind K, and e [M] (linear_w4.hip).
void launch_w4_halves(const W4Args& p, int Kp, uint4* xh, int32_t* xe, hipStream_t s);

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

// Eight codes of a dword as (q - z) 2^-9 in fp16, exact, in the column order of
// half_order; zero: -z 2^-9.
__device__ __forceinline__ f16x2_t zero_f16(float z) {
  const _Float16 v = (_Float16)(-0x1p-9f * z);
  return f16x2_t{v, v};
}
__device__ __forceinline__ f16x8_t codes_f16(uint32_t d, f16x2_t zero) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const f16x2_t one = {(_Float16)0x1p15f, (_Float16)0x1p15f};
  const f16x2_t one16 = {(_Float16)0x1p11f, (_Float16)0x1p11f};
  const uint32_t d8 = d >> 8;
  const auto low = [&](uint32_t v) {
    return __builtin_elementwise_fma(__builtin_bit_cast(f16x2_t, v & 0x000f000fu), one, zero);
  };
  const auto high = [&](uint32_t v) {
    return __builtin_elementwise_fma(__builtin_bit_cast(f16x2_t, v & 0x00f000f0u), one16, zero);
  };
  const u32x4 v = {__builtin_bit_cast(uint32_t, low(d)), __builtin_bit_cast(uint32_t, high(d)),
                   __builtin_bit_cast(uint32_t, low(d8)), __builtin_bit_cast(uint32_t, high(d8))};
  return __builtin_bit_cast(f16x8_t, v);
}

// The loads of a tile of 32 FM rows x 256 weight rows: four wavefronts, wavefront w
// with two tiles of 32 weight rows (with swiglu a tile of gates and the tile of their
// ups) and all the rows. A stage is 128 columns: x goes straight to one of two LDS
// buffers, the codes, which only one wavefront needs, to registers; both for the
// next stage while this one is multiplied. Scales and zero points go to LDS four
// groups at a time, a wavefront its own rows' (read per stage by the lanes that
// need them they took 60 of 277 us at 4096 x 8192 x 4096: 32 lines a load).
//   An LDS row of x is 256 bytes; 16-byte piece c of row r lies at c ^ (r & 15), so
// that a fragment's 32 rows reach all banks. Codes are loaded 16 rows x 64 bytes at
// a time; pieces() brings them to the lanes of their rows.
template <int G, bool SB, bool Z, int FM>
struct TileLoads {
  static constexpr int TM = 32 * FM, kBuf = TM * 256, NG = 128 / G, kPer = 4 / NG;
  static constexpr int kSet = 4096 * (Z ? 2 : 1);  // four groups of 256 rows, a dword each
  static constexpr int kBytes = 2 * kBuf + 2 * kSet;
  const W4Args& p;
  uint8_t* ring;
  uint32_t lds0;
  RowTile tile;
  int lane, l32, h, wave, n_out, groups, n0, stages, Kp;
  int64_t bank;
  const uint8_t* wb[2];  // (uniform bases and 32-bit offsets: registers are scarce)
  uint32_t wo[2][2], xo[2 * FM];
  const uint16_t* xb;

  // weight row of row r of the wavefront's tile j (rows past the last repeat it)
  __device__ __forceinline__ int row_of(int j, int r) const {
    const int n = n0 + r + (p.swiglu ? 0 : 32 * j);
    return (n < n_out ? n : n_out - 1) + (p.swiglu ? j * n_out : 0);
  }
  __device__ __forceinline__ TileLoads(const W4Args& args, uint8_t* lds, const RowTile& t, int tn,
                                       const uint16_t* xh, int padded_k)
      : p(args), ring(lds), lds0(lds_offset(lds)), tile(t), Kp(padded_k) {
    const int tid = threadIdx.x;
    lane = tid & 63;
    l32 = lane & 31;
    h = lane >> 5;
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    n_out = p.swiglu ? p.N / 2 : p.N;
    groups = p.K / G;
    n0 = p.swiglu ? tn * 128 + wave * 32 : tn * 256 + wave * 64;
    stages = Kp / kW4Stage;
    bank = (int64_t)tile.e * p.N;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int n = n0 + (p.swiglu ? 0 : 32 * j), first = n < n_out ? n : n_out - 1;
      wb[j] = p.w + (bank + first + (p.swiglu ? j * n_out : 0)) * (p.K / 2);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * i + (lane & 15);
        wo[j][i] = (uint32_t)(r < n_out - first ? r : n_out - 1 - first) * (uint32_t)(p.K / 2);
      }
    }
    // this thread's pieces of a stage, rows 16 apart (which leaves the swizzle alone)
    const int r0 = tid >> 4;
    xb = xh + tile.r0 * Kp;
#pragma unroll
    for (int i = 0; i < 2 * FM; ++i) {
      const int r = r0 + 16 * i < tile.rows ? r0 + 16 * i : tile.rows - 1;
      xo[i] = 2u * ((uint32_t)r * (uint32_t)Kp + 8 * ((tid & 15) ^ r0));
    }
  }
  // stage kb's x and, where it is the first of four groups, their scales
  __device__ __forceinline__ void issue(int kb) const {
#pragma unroll
    for (int i = 0; i < 2 * FM; ++i)
      lds16(lds0 + 1024 * wave + (kb & 1) * kBuf + 4096 * i, xb + kb * kW4Stage, xo[i]);
    if (kb % kPer != 0) return;
    // lane: row 16 i + lane % 16, group lane / 16
    const int g = 4 * (kb / kPer) + (lane >> 4);
    const uint32_t to = lds0 + 2 * kBuf + (kb / kPer & 1) * kSet + 1024 * wave;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at =
          (bank + row_of(i / 2, 16 * (i & 1) + (lane & 15))) * groups + (g < groups ? g : groups - 1);
      lds4_at<SB ? 2 : 4>(to + 256 * i, static_cast<const uint8_t*>(p.ws) + at * (SB ? 2 : 4));
      if (Z) lds4_at<1>(to + 4096 + 256 * i, p.wz + at);
    }
  }
  __device__ __forceinline__ void fetch(int kb, uint4 (&c)[2][2]) const {
    const int col = kb * kW4Stage + 32 * (lane >> 4);  // (x is zero behind K: any code will do)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) c[j][i] = ld16(wb[j] + (wo[j][i] + (col < p.K ? col : 0) / 2));
  }
  // scale and zero point of the lane's weight row of tile j, group g of the stage
  __device__ __forceinline__ void scale_of(int kb, int j, int g, float& s, float& z) const {
    const uint8_t* at = ring + 2 * kBuf + (kb / kPer & 1) * kSet + 1024 * wave +
                        256 * (2 * j + (l32 >> 4)) + 64 * (NG * (kb % kPer) + g) + 4 * (l32 & 15);
    s = __uint_as_float(*reinterpret_cast<const uint32_t*>(at) << (SB ? 16 : 0));
    z = Z ? (float)*reinterpret_cast<const uint32_t*>(at + 4096) : 8.f;
  }
  // [rows 0 .. 15: pieces 0 .. 3], [rows 16 .. 31: pieces 0 .. 3] by 16 lanes, to pieces
  // 2 h and 2 h + 1 of row l32
  static __device__ __forceinline__ void pieces(uint4 (&c)[2]) {
    uint32_t a[4] = {c[0].x, c[0].y, c[0].z, c[0].w}, b[4] = {c[1].x, c[1].y, c[1].z, c[1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto s = __builtin_amdgcn_permlane16_swap(a[i], b[i], false, false);
      a[i] = s[0];
      b[i] = s[1];
    }
    c[0] = make_uint4(a[0], a[1], a[2], a[3]);
    c[1] = make_uint4(b[0], b[1], b[2], b[3]);
  }
  // piece c of row 32 m + l32 of x
  __device__ __forceinline__ f16x8_t x_piece(int kb, int m, int c) const {
    return __builtin_bit_cast(
        f16x8_t, *reinterpret_cast<const uint4*>(ring + (kb & 1) * kBuf + m * 8192 + l32 * 256 +
                                                 16 * (c ^ (l32 & 15))));
  }
};

// bf16 output. What bounds it is the matrix unit and the vector unit that makes its
// weights, side by side: 4096 x 8192 x 4096 takes 252 us (1.09 PFLOP/s), of whose
// cycles matrix instructions fill 54 %, vector instructions 41 % and LDS 16 %.
// Lane l holds columns 64 h .. 64 h + 63 of row l % 32 of either operand,
// h = l / 32; instruction i takes eight of them.
template <int G, bool SB, bool Z, int FM>
__global__ __launch_bounds__(256, 2) void w4_tile(W4Args p, const uint16_t* __restrict__ xh,
                                                  const int32_t* __restrict__ xe, int Kp,
                                                  int tiles_m, int tiles_n) {
  using L = TileLoads<G, SB, Z, FM>;
  constexpr int TM = 32 * FM, NS = G == 32 ? 2 : 1;  // NS: scales of a lane's 64 columns
  __shared__ __attribute__((aligned(1024))) uint8_t lds[L::kBytes];
  int tm, tn;
  w4_tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const RowTile tile = find_tile<TM>(p, tm);
  if (tile.rows <= 0) return;
  const L ld(p, lds, tile, tn, xh, Kp);
  const int lane = ld.lane, l32 = ld.l32, h = ld.h, wave = ld.wave, groups = ld.groups;
  uint4 next[2][2];
  ld.issue(0);
  ld.fetch(0, next);
  // The weight rows' powers of two: eight lanes a row look for its largest scale, and
  // leave it in the second buffer of scales, which is not in use yet.
  float* tops = reinterpret_cast<float*>(lds + 2 * L::kBuf + L::kSet + 1024 * wave);
  {
    using Scale = std::conditional_t<SB, uint16_t, uint32_t>;
    float top[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t at = (ld.bank + ld.row_of(i / 4, 8 * (i % 4) + (lane >> 3))) * groups;
      const Scale* sp = static_cast<const Scale*>(p.ws) + at;
      top[i] = 0.f;
      for (int g = lane & 7; g < groups; g += 8)
        top[i] = fmaxf(top[i], fabsf(__uint_as_float((uint32_t)sp[g] << (SB ? 16 : 0))));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      top[i] = fmaxf(top[i], dpp_f<kDppXor1>(top[i]));
      top[i] = fmaxf(top[i], dpp_f<kDppXor2>(top[i]));
      top[i] = fmaxf(top[i], dpp_f<kDppHalfMirror>(top[i]));
      if ((lane & 7) == 0) tops[8 * i + (lane >> 3)] = top[i];
    }
  }
  wave_lds_fence();
  int en[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float m = tops[32 * j + l32];
    en[j] = m > 0.f ? __builtin_amdgcn_frexp_expf(m) - 6 : 0;  // the weights' power of two
  }
  f32x16 acc[2][FM];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[j][m][v] = 0.f;
#pragma unroll 1
  for (int kb = 0; kb < ld.stages; ++kb) {
    w4_wait<0>();
    lds_barrier();  // everyone's pieces are there, and the other buffer has been read
    uint4 c[2][2] = {{next[0][0], next[0][1]}, {next[1][0], next[1][1]}};
    if (kb + 1 < ld.stages) {
      ld.issue(kb + 1);
      ld.fetch(kb + 1, next);
    }
    f16x8_t S[2][NS];
    f16x2_t zero[2][NS];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        float sv, zv;
        ld.scale_of(kb, j, G == 128 ? 0 : G == 64 ? h : 2 * h + i, sv, zv);
        const _Float16 v = (_Float16)__builtin_ldexpf(sv, 9 - en[j]);
        S[j][i] = f16x8_t{v, v, v, v, v, v, v, v};
        zero[j][i] = zero_f16(zv);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) L::pieces(c[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f16x8_t w[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 q = c[j][i / 4];
        const uint32_t d[4] = {q.x, q.y, q.z, q.w};
        constexpr int kEach = 8 / NS;
        w[j] = codes_f16(d[i % 4], zero[j][i / kEach]) * S[j][i / kEach];
      }
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const f16x8_t x = ld.x_piece(kb, m, 8 * h + i);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[j][m] = __builtin_amdgcn_mfma_f32_32x32x16_f16(w[j], x, acc[j][m], 0, 0, 0);
      }
    }
  }
  // Value v of a lane: weight row 8 (v / 4) + 4 h + v % 4, row l32 of x. Rows go out
  // through LDS (the buffers are free) in 16-byte pieces: a lane's four features are
  // half a piece.
  lds_barrier();
  const int width = p.swiglu ? 64 : 128;  // bytes of a wavefront's output row
  uint8_t* mine = lds + wave * (FM * 4096);
  int er[FM];
#pragma unroll
  for (int m = 0; m < FM; ++m)
    er[m] = xe[tile.r0 + (32 * m + l32 < tile.rows ? 32 * m + l32 : tile.rows - 1)];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int f = 8 * b + 4 * h;
    int e[2][4];
    float bias[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        e[j][v] = __shfl(en[j], f + v);
        bias[j][v] = p.bias ? p.bias[ld.bank + ld.row_of(j, f + v)] : 0.f;
      }
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const int r = 32 * m + l32;
      float y[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          y[j][v] = __builtin_ldexpf(acc[j][m][4 * b + v], e[j][v] + er[m]) + bias[j][v];
      const auto put = [&](int piece, const float (&v)[4]) {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<bf16x4*>(mine + r * width + 16 * piece + 8 * h) =
            bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
      };
      if (p.swiglu) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = w4_silu(y[0][i]) * y[1][i];
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
    const int r = i / per, c = i % per, n = ld.n0 + 8 * c;
    if (r >= tile.rows) break;
    const uint4 v = *reinterpret_cast<const uint4*>(
        mine + r * width + 16 * (p.swiglu ? c ^ ((r >> 1) & 3) : c ^ (r & 7)));
    uint16_t* at = out + (tile.r0 + r) * p.ld_out + n;
    if (p.out_vec && n + 8 <= ld.n_out) {
      *reinterpret_cast<uint4*>(at) = v;
    } else {
      const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (n + k < ld.n_out) at[k] = (uint16_t)(d[k / 2] >> (16 * (k & 1)));
    }
  }
}

// fp32 output: the same rows of x, and weights that are the whole numbers q - z times
// 2^-9, exact in fp16; a group's sum is scaled in fp32 as it is added. So a group has
// to be whole instructions: instruction i takes columns 16 i .. 16 i + 15, eight a
// half wavefront (one more exchange of the codes' dwords). A row tile's products of
// one group follow each other in one accumulator. The codes are the B operand: a lane
// holds one output feature, whose scale it reads itself, and 32 lanes store a line.
//   The multiply-adds on each sum and group bound it: one group of 32 columns is two
// products of 32 cycles and 16 multiply-adds of 4. 4096 x 8192 x 4096, a call: 310 us in
// groups of 128 (0.89 PFLOP/s), 405 in groups of 32; 338 and 494 with zero points.
template <int G, bool SB, bool Z, int FM>
__global__ __launch_bounds__(256, 2) void w4_tile_exact(W4Args p, const uint16_t* __restrict__ xh,
                                                        const int32_t* __restrict__ xe, int Kp,
                                                        int tiles_m, int tiles_n) {
  using L = TileLoads<G, SB, Z, FM>;
  constexpr int TM = 32 * FM, NG = 128 / G, NI = G / 16;  // NI: instructions of a group
  __shared__ __attribute__((aligned(1024))) uint8_t lds[L::kBytes];
  int tm, tn;
  w4_tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
  const RowTile tile = find_tile<TM>(p, tm);
  if (tile.rows <= 0) return;
  const L ld(p, lds, tile, tn, xh, Kp);
  const int l32 = ld.l32, h = ld.h;
  uint4 next[2][2];
  ld.issue(0);
  ld.fetch(0, next);
  f32x16 acc[2][FM];
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[j][m][v] = 0.f;
#pragma unroll 1
  for (int kb = 0; kb < ld.stages; ++kb) {
    w4_wait<0>();
    lds_barrier();  // everyone's pieces are there, and the other buffer has been read
    uint4 c[2][2] = {{next[0][0], next[0][1]}, {next[1][0], next[1][1]}};
    if (kb + 1 < ld.stages) {
      ld.issue(kb + 1);
      ld.fetch(kb + 1, next);
    }
    // dword 2 i + h of the row for instruction i
    uint32_t d[2][8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      L::pieces(c[j]);
      const uint32_t a[8] = {c[j][0].x, c[j][0].y, c[j][0].z, c[j][0].w,
                             c[j][1].x, c[j][1].y, c[j][1].z, c[j][1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const auto s = __builtin_amdgcn_permlane32_swap(a[2 * i], a[2 * i + 1], false, false);
        d[j][i] = s[0];
        d[j][i + 4] = s[1];
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float s[2];
      f16x8_t w[2][NI];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float z;
        ld.scale_of(kb, j, g, s[j], z);
        const f16x2_t zero = zero_f16(z);
#pragma unroll
        for (int i = 0; i < NI; ++i) w[j][i] = codes_f16(d[j][g * NI + i], zero);
      }
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        f32x16 sum[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) sum[j][v] = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const f16x8_t x = ld.x_piece(kb, m, 2 * (g * NI + i) + h);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            sum[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, w[j][i], sum[j], 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) acc[j][m][v] = fmaf(s[j], sum[j][v], acc[j][m][v]);
      }
    }
  }
  // value v of a lane: row 8 (v / 4) + 4 h + v % 4 of x, weight row l32
  float bias[2] = {0.f, 0.f};
  if (p.bias) {
#pragma unroll
    for (int j = 0; j < 2; ++j) bias[j] = p.bias[ld.bank + ld.row_of(j, l32)];
  }
#pragma unroll
  for (int m = 0; m < FM; ++m)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int r = 32 * m + 8 * (v / 4) + 4 * h + v % 4;
      if (r >= tile.rows) continue;
      const int e = xe[tile.r0 + r] + 9;
      float y[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) y[j] = __builtin_ldexpf(acc[j][m][v], e) + bias[j];
      if (p.swiglu) {
        if (ld.n0 + l32 < ld.n_out) w4_store(p, tile.r0 + r, ld.n0 + l32, w4_silu(y[0]) * y[1]);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (ld.n0 + 32 * j + l32 < ld.n_out)
            w4_store(p, tile.r0 + r, ld.n0 + 32 * j + l32, y[j]);
      }
    }
}

// ---------------------------------------------------------------- host side --
// Row tiles of at most TM rows: every expert's last one may be short.
inline int64_t row_tiles(const W4Args& p, int TM) {
  return p.offsets ? p.M / TM + (p.M < p.E ? p.M : p.E) : (p.M + TM - 1) / TM;
}

// Columns that the stream multiplies for each strip: those of all its wavefronts' units
// (launch_w4), whether K fills them or not, once more for each pass.
constexpr int kW4Pass = 4096;
inline int w4_span(int K) {
  if (K <= 2048) return K <= 768 ? 768 : K <= 1024 ? 1024 : 2048;
  return (K + kW4Pass - 1) / kW4Pass * kW4Pass;
}

// Which kernel a product runs on: the one that is reckoned to take less time (us on one
// MI355X, weights in no cache). The weights of the experts that can have a row, read
// once, take W = E N K / 10^7.
//   stream  8 + 5.4e-9 (M + 10 (E - 1)) N span + 0.75 W: E short tiles; the second term
//           twice where x is read again for every pass. 4096 x 4096, 128 / 512 / 1024 rows:
//           21 / 54 / 99; 128 experts of 2048 x 2048, 32 / 64 / 96 rows each: 143 / 233 /
//           331; 4096 rows, 4096 x 32: 92; 1024 rows, 4096 x 128: 23; 256 rows, 4096 x 4096
//           / 4128: 27 / 103; 103 rows of 222 experts of 8026 x 192: 62
//   tiles   12.5 + 2.5e-9 (M + 32 E) N K + W, at least 8 + 1.45 a stage + W; fp32 output
//           2.9e-9 (M + 48 E): E short tiles. The same sizes: 54 / 57 / 63, fp32 52 / 56 /
//           68; 146 / 190 / 241, fp32 169 / 238 / 284; 20, fp32 34; 14, 17; 44 / 69, 43 /
//           58; fp32 34
// (Of 848 products of 16 to 16384 rows, 64 to 8192 features and 32 to 8192 columns it
// takes one that is over 1.1 times as slow as the other in 28, 1.45 times at most; most of
// those are short, where the host's 2.5 us for a second launch count.)
enum W4Form { kW4Stream, kW4Tiles };
inline W4Form w4_form(int64_t M, int E, int N, int K, bool bf16) {
  const double experts = (double)(M < E ? M : E), NK = (double)N * K, W = experts * NK * 1e-7;
  const double stream =
      8.0 + (K > kW4Pass ? 10.8e-9 : 5.4e-9) * (M + 10 * (experts - 1)) * N * w4_span(K) + 0.75 * W;
  const double busy = 12.5 + (bf16 ? 2.5e-9 * (M + 32 * experts) : 2.9e-9 * (M + 48 * experts)) * NK;
  const double stages = 8.0 + 1.45 * ((K + kW4Stage - 1) / kW4Stage);
  return stream <= W + (busy > stages ? busy : stages) ? kW4Stream : kW4Tiles;
}

inline int w4_padded(int K) { return (K + kW4Stage - 1) / kW4Stage * kW4Stage; }
inline size_t w4_al256(size_t n) { return (n + 255) / 256 * 256; }

// Eight wavefronts of 20 KiB of LDS a compute unit, in workgroups of W.
template <int G, bool SB, bool Z, int W, int UW, bool LONG>
void launch_stream(const W4Args& p, hipStream_t s) {
  const int strips = ((p.swiglu ? p.N / 2 : p.N) + 15) / 16;
  const int64_t most = row_tiles(p, 16) * strips;
  constexpr int kGrid = kW4Units * 8 / W;
  w4_stream<G, SB, Z, W, UW, 20 * W - 1, LONG>
      <<<(unsigned)(most < kGrid ? most : kGrid), 64 * W, 0, s>>>(p);
}

// Tiles of 32 FM rows whose rounds of workgroups cost least. A stage of a round takes,
// with two workgroups on every compute unit, 1.55 us at FM = 1, 2.3 at 2, 4.0 at 4; 1.1,
// 1.25 and 1.95 with one at most (fp32 output: 1.6 and 2.35, 1.2 and 1.3).
// By expert, half a tile for each is reckoned as its short one.
template <bool EXACT>
int best_tile(const W4Args& p) {
  const int cols = p.swiglu ? 128 : 256;
  const double strips = ((p.swiglu ? p.N / 2 : p.N) + cols - 1) / cols;
  const double full[2][3] = {{1.55, 2.3, 4.0}, {1.6, 2.35, 0}},
               alone[2][3] = {{1.1, 1.25, 1.95}, {1.2, 1.3, 0}};
  int best = 1;
  double least = 0;
  for (int i = 0; i < (EXACT ? 2 : 3); ++i) {
    const int TM = 32 << i;
    const double tiles = p.offsets ? (double)p.M / TM + 0.5 * (p.M < p.E ? p.M : p.E)
                                   : (double)((p.M + TM - 1) / TM);
    const double groups = tiles * strips, slots = 2.0 * kW4Units;
    const double cost = groups <= kW4Units ? alone[EXACT][i]
                                           : full[EXACT][i] * (groups <= slots ? 1.0 : groups / slots);
    if (i == 0 || cost < least) {
      least = cost;
      best = 1 << i;
    }
  }
  return best;
}

template <int G, bool SB, bool Z, int FM, bool EXACT>
void launch_tile(const W4Args& p, const uint16_t* xh, const int32_t* xe, hipStream_t s) {
  const int n_out = p.swiglu ? p.N / 2 : p.N, cols = p.swiglu ? 128 : 256;
  const int tm = (int)row_tiles(p, 32 * FM), tn = (n_out + cols - 1) / cols;
  const unsigned grid = (unsigned)((int64_t)tm * tn);
  if constexpr (EXACT)
    w4_tile_exact<G, SB, Z, FM><<<grid, 256, 0, s>>>(p, xh, xe, w4_padded(p.K), tm, tn);
  else
    w4_tile<G, SB, Z, FM><<<grid, 256, 0, s>>>(p, xh, xe, w4_padded(p.K), tm, tn);
}

template <int G, bool SB, bool Z>
void launch_w4(const W4Args& p, void* workspace, hipStream_t s) {
  const W4Form form = w4_form(p.M, p.E, p.N, p.K, p.out_bf16);
  if (form == kW4Stream) {
    // wavefronts and units that cover K with the fewest idle ones (1024 columns: 2 x 4 37
    // us, 4 x 2 41, 8 x 1 50; 2048: 4 x 4 30, 8 x 2 36; 4096: 8 x 4 64, 16 x 2 72)
    if (p.K <= 768) return launch_stream<G, SB, Z, 2, 3, false>(p, s);
    if (p.K <= 1024) return launch_stream<G, SB, Z, 2, 4, false>(p, s);
    if (p.K <= 2048) return launch_stream<G, SB, Z, 4, 4, false>(p, s);
    if (p.K <= kW4Pass) return launch_stream<G, SB, Z, 8, 4, false>(p, s);
    return launch_stream<G, SB, Z, 8, 4, true>(p, s);
  }
  const int Kp = w4_padded(p.K);
  uint4* xh = static_cast<uint4*>(workspace);
  int32_t* xe = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) +
                                           w4_al256((size_t)p.M * Kp * 2));
  launch_w4_halves(p, Kp, xh, xe, s);
  const uint16_t* rows = reinterpret_cast<const uint16_t*>(xh);
  if (!p.out_bf16)
    return best_tile<true>(p) == 1 ? launch_tile<G, SB, Z, 1, true>(p, rows, xe, s)
                                   : launch_tile<G, SB, Z, 2, true>(p, rows, xe, s);
  switch (best_tile<false>(p)) {
    case 1: return launch_tile<G, SB, Z, 1, false>(p, rows, xe, s);
    case 2: return launch_tile<G, SB, Z, 2, false>(p, rows, xe, s);
    default: return launch_tile<G, SB, Z, 4, false>(p, rows, xe, s);
  }
}

template <int G>
void launch_w4_group(const W4Args& p, void* workspace, hipStream_t s) {
  if (p.ws_bf16)
    p.wz ? launch_w4<G, true, true>(p, workspace, s) : launch_w4<G, true, false>(p, workspace, s);
  else
    p.wz ? launch_w4<G, false, true>(p, workspace, s) : launch_w4<G, false, false>(p, workspace, s);
}

}  // namespace moe
