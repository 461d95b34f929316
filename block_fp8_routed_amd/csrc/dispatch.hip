// dispatch.hip — the rows of a batch sorted by expert (moe_dispatch), weighted
// back (moe_combine), and the gradients of both.
//
// Slot s = t k + j is the j-th choice of token t. With key(s) = (expert, s) a
// slot's row is the number of slots of a smaller key: the stable sort by expert
// that moe_permute describes. A slot whose expert is outside [0, experts) has no
// row (inv = -1) and takes no part.
//   dispatch           rows[inv[s]] = x[t]
//   dispatch_backward  dx[t]  = sum_j d_rows[inv[t,j]]
//   combine            out[t] = sum_j g[t,j] y[inv[t,j]] (+ shared[t])
//   combine_backward   d_y[inv[t,j]] = g[t,j] d_out[t],  d_g[t,j] = <d_out[t], y[inv[t,j]]>
// All are bound by the bytes of the rows: a token's own row is read (or written)
// once, its k others written (or read) once. So every kernel goes by token, with
// the k rows' accesses of a thread's columns in flight together; sums are fp32
// in the order of the slots, one rounding at the end. Where a large copy moves 5.1
// TB/s, reads alone 6: copies of a gradient of 369 MB take 63 us (5.9 TB/s), those of
// a prompt of 369 MB 71 to 76 (5), combine of 403 MB 68 (5.9), combine_backward of 286
// MB 59 (4.8).
#include "device.hpp"
#include "layer.hpp"
#include "permute.hpp"

#include <type_traits>

namespace moe {

// ------------------------------------------------------------------ elements --
// N values of a row at p, which is aligned to N elements or 16 bytes.
template <class T, int N>
struct Pack {
  T v[N];
};
template <class T, int N>
__device__ __forceinline__ Pack<T, N> ld_pack(const T* p) {
  constexpr int B = sizeof(T) * N;
  constexpr int A = B < 16 ? B : 16;
  typedef unsigned char bytes __attribute__((ext_vector_type(A), aligned(A)));
  Pack<T, N> r;
#pragma unroll
  for (int i = 0; i < B / A; ++i) {
    const bytes b = __builtin_nontemporal_load(reinterpret_cast<const bytes*>(p) + i);
    __builtin_memcpy(reinterpret_cast<char*>(r.v) + i * A, &b, A);
  }
  return r;
}
template <class T, int N>
__device__ __forceinline__ void st_pack(T* p, const Pack<T, N>& r) {
  constexpr int B = sizeof(T) * N;
  constexpr int A = B < 16 ? B : 16;
  typedef unsigned char bytes __attribute__((ext_vector_type(A), aligned(A)));
#pragma unroll
  for (int i = 0; i < B / A; ++i) {
    bytes b;
    __builtin_memcpy(&b, reinterpret_cast<const char*>(r.v) + i * A, A);
    __builtin_nontemporal_store(b, reinterpret_cast<bytes*>(p) + i);
  }
}

constexpr int kDispSmall = 4096;   // up to this many slots each workgroup ranks its own token's
constexpr int kDispChunk = 1024;   // slots a placing workgroup takes, at least
constexpr int kDispChunks = 64;    // placing workgroups at most

// -------------------------------------------------------- one launch (small) --
// Workgroup t < T ranks the slots of token t against all others and copies its
// row; workgroup T writes offsets. No workgroup needs another's result: a rank is
// k comparisons a slot (wave-wide, counted by ballots), which for up to
// kDispSmall slots costs less than a second launch (512 tokens of 8 slots 11 us, 513
// in three launches 12; one token 4.2). blockIdx.y: column chunks.
template <class T, int N>
__global__ __launch_bounds__(256) void dispatch_small(
    const T* __restrict__ x, int64_t ld_x, const int32_t* __restrict__ topk, int tokens, int H,
    int k, int E, T* __restrict__ rows, int64_t ld_rows, int32_t* __restrict__ offsets,
    int32_t* __restrict__ pair, int32_t* __restrict__ inv) {
  constexpr int kNone = 0x7fffffff;
  static_assert(kDispSmall <= 4096 && kMaxExperts <= 1 << 18, "a key is expert * 4096 + slot");
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int TK = tokens * k, t = blockIdx.x;
  if (t == tokens) {
    if (blockIdx.y > 0) return;
    __shared__ int32_t cnt[kMaxExperts];
    __shared__ int32_t tmp[64];
    for (int e = tid; e < kMaxExperts; e += 256) cnt[e] = 0;
    __syncthreads();
    for (int s = tid; s < TK; s += 256) {
      const int e = topk[s];
      if ((unsigned)e < (unsigned)E) atomicAdd(&cnt[e], 1);
    }
    __syncthreads();
    constexpr int PER = kMaxExperts / 256;
    int c[PER], sum[1] = {0}, first[1], total[1];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = cnt[PER * tid + i];
      sum[0] += c[i];
    }
    block_excl_scan<4, 1>(sum, first, total, tmp);
    int run = first[0];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (PER * tid + i < E) offsets[PER * tid + i] = run;
      run += c[i];
    }
    if (tid == 0) offsets[E] = total[0];
    return;
  }
  __shared__ int32_t part[4][kMaxTopK + 1];
  // (the row's load goes out before the ranks are known)
  const int c = (blockIdx.y * 256 + tid) * N;
  Pack<T, N> v;
  if (c < H) v = ld_pack<T, N>(x + t * ld_x + c);
  int mine[kMaxTopK];  // the keys of the token's own slots (uniform)
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    const int s = t * k + (j < k ? j : 0);
    const int e = topk[s];
    mine[j] = (unsigned)e < (unsigned)E ? e * 4096 + s : kNone;
  }
  int below[kMaxTopK], valid = 0;
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) below[j] = 0;
  for (int s0 = 0; s0 < TK; s0 += 256) {
    const int s = s0 + tid;
    const int e = s < TK ? topk[s] : -1;
    const int key = (unsigned)e < (unsigned)E ? e * 4096 + s : kNone;
    valid += __popcll(__ballot(key != kNone));
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j)
      if (j < k) below[j] += __popcll(__ballot(key < mine[j]));
  }
  if (lane == 0) {
#pragma unroll
    for (int j = 0; j < kMaxTopK; ++j) part[w][j] = below[j];
    part[w][kMaxTopK] = valid;
  }
  __syncthreads();
  const int sum = part[0][lane & 15] + part[1][lane & 15] + part[2][lane & 15] + part[3][lane & 15];
  if (blockIdx.y == 0 && tid < k) {
    const int s = t * k + tid;
    const int total = part[0][kMaxTopK] + part[1][kMaxTopK] + part[2][kMaxTopK] + part[3][kMaxTopK];
    const bool ok = (unsigned)topk[s] < (unsigned)E;
    inv[s] = ok ? sum : -1;
    if (ok) pair[sum] = s;
    if (s >= total) pair[s] = -1;
  }
  if (c >= H) return;
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j)
    if (j < k && mine[j] != kNone)
      st_pack<T, N>(rows + (int64_t)(part[0][j] + part[1][j] + part[2][j] + part[3][j]) * ld_rows + c, v);
}

// ------------------------------------------------------------ three launches --
// dispatch_count: workgroup b counts the slots of its chunk by expert. (2.5 to 4.6 us,
// dispatch_place 5 to 6.5.)
__global__ __launch_bounds__(1024) void dispatch_count(const int32_t* __restrict__ topk, int64_t TK,
                                                       int64_t per, int E,
                                                       int32_t* __restrict__ counts) {
  __shared__ int32_t cnt[kMaxExperts];
  const int tid = threadIdx.x;
  const int64_t lo = blockIdx.x * per, hi = lo + per < TK ? lo + per : TK;
  if (tid < E) cnt[tid] = 0;
  __syncthreads();
  for (int64_t s = lo + tid; s < hi; s += 1024) {
    const int e = topk[s];
    if ((unsigned)e < (unsigned)E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (tid < E) counts[(int64_t)blockIdx.x * E + tid] = cnt[tid];
}

// dispatch_place: workgroup b places the slots of its chunk. Thread e sums expert
// e's counts over all chunks and over those before b; a scan over the experts
// gives their first rows. Wavefront w then takes a consecutive part of the chunk:
// it counts the part (LDS), gets its own first rows by a prefix over the
// wavefronts, and walks its slots in order, lanes of one expert ranked by ballots.
__global__ __launch_bounds__(1024) void dispatch_place(
    const int32_t* __restrict__ topk, int64_t TK, int64_t per, int E,
    const int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ pair,
    int32_t* __restrict__ inv) {
  extern __shared__ int32_t next[];  // [16][E] the wavefronts' next rows
  __shared__ int32_t tmp[64];
  constexpr int W = 16;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t lo = blockIdx.x * per, hi = lo + per < TK ? lo + per : TK;
  const int64_t wper = (per / W + 63) / 64 * 64;
  const int64_t wlo = lo + w * wper < hi ? lo + w * wper : hi;
  const int64_t whi = wlo + wper < hi ? wlo + wper : hi;
  for (int i = tid; i < W * E; i += 1024) next[i] = 0;
  __syncthreads();
  for (int64_t s = wlo + lane; s < whi; s += 64) {
    const int e = topk[s];
    if ((unsigned)e < (unsigned)E) atomicAdd(&next[w * E + e], 1);
  }
  int all[1] = {0}, first[1], total[1], before = 0;
  if (tid < E) {
#pragma unroll 8
    for (int b = 0; b < (int)gridDim.x; ++b) {
      const int c = counts[(int64_t)b * E + tid];
      if (b < (int)blockIdx.x) before += c;
      all[0] += c;
    }
  }
  block_excl_scan<W, 1>(all, first, total, tmp);  // (its barriers end the counting too)
  if (blockIdx.x == 0) {
    if (tid < E) offsets[tid] = first[0];
    if (tid == 0) offsets[E] = total[0];
  }
  for (int64_t s = lo + tid; s < hi; s += 1024)
    if (s >= total[0]) pair[s] = -1;
  if (tid < E) {
    int run = first[0] + before;
    for (int ww = 0; ww < W; ++ww) {
      const int c = next[ww * E + tid];
      next[ww * E + tid] = run;
      run += c;
    }
  }
  __syncthreads();
  const int bits = E > 1 ? 32 - __clz(E - 1) : 0;
  for (int64_t s0 = wlo; s0 < whi; s0 += 64) {
    const int64_t s = s0 + lane;
    const int got = s < whi ? topk[s] : -1;
    const bool ok = (unsigned)got < (unsigned)E;
    const int e = ok ? got : 0;
    uint64_t peers = __ballot(ok);
    for (int b = 0; b < bits; ++b) {
      const bool bit = (e >> b) & 1;
      const uint64_t m = __ballot(ok && bit);
      peers &= bit ? m : ~m;
    }
    const int rank = __popcll(peers & ((1ull << lane) - 1ull));
    const int row = next[w * E + e] + rank;
    wave_lds_fence();  // every lane has read before a first lane moves the counter on
    if (ok && rank == 0) next[w * E + e] = row + __popcll(peers);
    wave_lds_fence();
    if (s < whi) inv[s] = ok ? row : -1;
    if (ok) pair[row] = (int32_t)s;
  }
}

// ------------------------------------------------------------- rows by token --
// W wavefronts a token (4: one column chunk of 256 N a workgroup, blockIdx.y; 1:
// four tokens a workgroup, rows of at most 64 N columns). A token's slots with a
// row are the set bits of a mask; lane j holds slot j's row.
template <int W>
struct Place {
  int64_t t;
  int c;  // thread's columns, over N
};
template <int W>
__device__ __forceinline__ Place<W> place_of() {
  if (W == 1) {
    // (uniform in a wavefront: kept in scalar registers)
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    return {(int64_t)blockIdx.x * 4 + w, (int)(threadIdx.x & 63)};
  }
  return {(int64_t)blockIdx.x, (int)(blockIdx.y * 256 + threadIdx.x)};
}
__device__ __forceinline__ int next_slot(uint64_t& m) {
  const int j = __builtin_ctzll(m);
  m &= m - 1;
  return j;
}

template <class T, int N, int W>
__global__ __launch_bounds__(256) void dispatch_rows(const T* __restrict__ x, int64_t ld_x,
                                                     int64_t tokens, int H, int k,
                                                     const int32_t* __restrict__ inv,
                                                     T* __restrict__ rows, int64_t ld_rows) {
  const Place<W> p = place_of<W>();
  const int c = p.c * N;
  if (p.t >= tokens) return;
  const int lane = threadIdx.x & 63;
  const int row = lane < k ? inv[p.t * k + lane] : -1;
  uint64_t m = __ballot(row >= 0);
  const bool in = c < H;
  // (lanes past H stay, with column 0: readlane needs every lane's row)
  const Pack<T, N> v = ld_pack<T, N>(x + p.t * ld_x + (in ? c : 0));
  while (m) {
    const int r = __builtin_amdgcn_readlane(row, next_slot(m));
    if (in) st_pack<T, N>(rows + (int64_t)r * ld_rows + c, v);
  }
}

// out[t] = sum_j g[t,j] y[inv[t,j]] (+ shared[t]); gates null: all 1 (the
// gradient of dispatch). B rows are requested before the first is added.
template <class O, class T, int N, int W>
__global__ __launch_bounds__(256) void combine_rows(
    const T* __restrict__ y, int64_t ld_y, int64_t nrows, const float* __restrict__ gates,
    const int32_t* __restrict__ inv, const T* __restrict__ shared, int64_t ld_s, int64_t tokens,
    int H, int k, O* __restrict__ out, int64_t ld_out) {
  const Place<W> p = place_of<W>();
  if (p.t >= tokens) return;
  const int lane = threadIdx.x & 63;
  const int row = lane < k ? inv[p.t * k + lane] : -1;
  const float gate = lane < k && gates ? gates[p.t * k + lane] : 1.f;
  uint64_t m = __ballot(row >= 0 && row < nrows);
  // (lanes past H stay, with column 0: readlane needs every lane's row and gate)
  const bool in = p.c * N < H;
  const int c = in ? p.c * N : 0;
  constexpr int B = sizeof(T) * N > 16 ? 4 : 8;
  float a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = 0.f;
  while (m) {
    Pack<T, N> v[B];
    float g[B];
    int n = 0;
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (m) {
        const int j = next_slot(m);
        const int r = __builtin_amdgcn_readlane(row, j);
        g[b] = readlane_f(gate, j);
        v[b] = ld_pack<T, N>(y + (int64_t)r * ld_y + c);
        n = b + 1;
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
      if (b < n) {
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] = fmaf(g[b], (float)v[b].v[i], a[i]);
      }
    }
  }
  if (shared) {
    const Pack<T, N> v = ld_pack<T, N>(shared + p.t * ld_s + c);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] += (float)v.v[i];
  }
  Pack<O, N> o;
#pragma unroll
  for (int i = 0; i < N; ++i) o.v[i] = (O)a[i];
  if (in) st_pack<O, N>(out + p.t * ld_out + c, o);
}

// The gradients of combine: W wavefronts walk a token's columns, 64 W N at a
// time, and hold the k partial sums of the gates' gradients; wavefronts are
// joined through LDS in their order.
template <class D, class T, int N, int W>
__global__ __launch_bounds__(256) void combine_grad(
    const D* __restrict__ d_out, int64_t ld_d, const T* __restrict__ y, int64_t ld_y,
    int64_t nrows, const float* __restrict__ gates, const int32_t* __restrict__ inv,
    int64_t tokens, int H, int k, T* __restrict__ d_y, int64_t ld_dy,
    float* __restrict__ d_gates) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t t = W == 1 ? (int64_t)blockIdx.x * 4 + w : (int64_t)blockIdx.x;
  if (t >= tokens) return;  // (W = 4: the whole workgroup, or none)
  const int row = lane < k ? inv[t * k + lane] : -1;
  const float gate = lane < k ? gates[t * k + lane] : 0.f;
  const uint64_t valid = __ballot(row >= 0 && row < nrows);
  float dot[kMaxTopK];
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) dot[j] = 0.f;
  for (int c0 = W == 1 ? 0 : w * 64 * N; c0 < H; c0 += 64 * W * N) {
    // (lanes past H stay, with column 0: readlane needs every lane's row and gate)
    const bool in = c0 + lane * N < H;
    const int c = in ? c0 + lane * N : 0;
    const Pack<D, N> d = ld_pack<D, N>(d_out + t * ld_d + c);
    constexpr int B = 4;
#pragma unroll
    for (int j0 = 0; j0 < kMaxTopK; j0 += B) {
      if (j0 >= k) continue;
      Pack<T, N> v[B];
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (valid >> (j0 + b) & 1)
          v[b] = ld_pack<T, N>(y + (int64_t)__builtin_amdgcn_readlane(row, j0 + b) * ld_y + c);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (valid >> (j0 + b) & 1) {
          const float g = readlane_f(gate, j0 + b);
          const int64_t at = (int64_t)__builtin_amdgcn_readlane(row, j0 + b) * ld_dy + c;
          Pack<T, N> o;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float next = fmaf((float)d.v[i], (float)v[b].v[i], dot[j0 + b]);
            dot[j0 + b] = in ? next : dot[j0 + b];
            o.v[i] = (T)(g * (float)d.v[i]);
          }
          if (in) st_pack<T, N>(d_y + at, o);
        }
      }
    }
  }
  __shared__ float part[4][kMaxTopK];
#pragma unroll
  for (int j = 0; j < kMaxTopK; ++j) {
    if (j >= k) continue;
    const float s = group_sum<64>(dot[j]);
    if (W == 1) {
      if (lane == 0) d_gates[t * k + j] = s;
    } else if (lane == 0) {
      part[w][j] = s;
    }
  }
  if (W == 1) return;
  __syncthreads();
  if ((int)threadIdx.x < k)
    d_gates[t * k + threadIdx.x] = ((part[0][threadIdx.x] + part[1][threadIdx.x]) +
                                    part[2][threadIdx.x]) + part[3][threadIdx.x];
}

// ---------------------------------------------------------------- host side --
// Tokens, hidden and the choice: fewer than 2^24 workgroups of 256 threads, and slots
// that fit an int32 with the last chunk's end.
static moe_status check_rows(int64_t tokens, int32_t H, int32_t k) {
  if (tokens < 0 || H <= 0 || k <= 0) return MOE_ERR_SHAPE;
  if (k > kMaxTopK || H > (1 << 20) || tokens >= ((int64_t)1 << 24) ||
      tokens * k > ((int64_t)1 << 27))
    return MOE_ERR_UNSUPPORTED;
  // workgroups of one token and 256 columns at least (and one token's for the offsets)
  if ((tokens + 1) * ((H + 255) / 256) >= ((int64_t)1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The largest N of 8, 4, 2, 1 elements (4 where all matrices are fp32: 16 bytes) at
// which every row of a matrix can be read: N divides the columns and the row
// distance, the base is aligned.
struct Shape {
  int n;
  Shape(int H, bool all_f32) : n(all_f32 ? 4 : 8) { limit(H); }
  void limit(int64_t v) {
    while (v % n != 0) n /= 2;
  }
  void matrix(const void* p, int64_t ld, moe_dtype t) {
    if (!p) return;
    const int size = t == MOE_BF16 ? 2 : 4;
    limit(ld);
    while (reinterpret_cast<uintptr_t>(p) % (n * size < 16 ? n * size : 16) != 0) n /= 2;
  }
};
static bool odd_elements(const void* p, moe_dtype t) {
  return reinterpret_cast<uintptr_t>(p) % (t == MOE_BF16 ? 2 : 4) != 0;
}
static bool odd4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; }
static bool is_dtype(moe_dtype t) { return t == MOE_F32 || t == MOE_BF16; }

template <class F>
static void with_type(moe_dtype t, F&& f) {
  if (t == MOE_BF16)
    f(static_cast<__bf16*>(nullptr));
  else
    f(static_cast<float*>(nullptr));
}
template <class F>
static void with_n(int n, F&& f) {
  switch (n) {
    case 8: return f(std::integral_constant<int, 8>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 2: return f(std::integral_constant<int, 2>{});
    default: return f(std::integral_constant<int, 1>{});
  }
}
// One wavefront a token where it covers the columns, else four and a grid of
// column chunks.
template <class F>
static void with_waves(int64_t tokens, int H, int n, F&& f) {
  if (H <= 64 * n)
    f(std::integral_constant<int, 1>{}, dim3((unsigned)((tokens + 3) / 4), 1));
  else
    f(std::integral_constant<int, 4>{},
      dim3((unsigned)tokens, (unsigned)((H + 256 * n - 1) / (256 * n))));
}

static size_t al256(size_t n) { return (n + 255) / 256 * 256; }
static int64_t chunk_slots(int64_t TK) {
  const int64_t per = (TK + kDispChunks - 1) / kDispChunks;
  return per < kDispChunk ? kDispChunk : (per + 1023) / 1024 * 1024;
}

static moe_status launch_combine_rows(const void* y, int64_t ld_y, int64_t nrows, moe_dtype yt,
                                      const float* gates, const int32_t* inv, const void* shared,
                                      int64_t ld_s, int64_t tokens, int H, int k, void* out,
                                      int64_t ld_out, moe_dtype ot, hipStream_t s) {
  Shape a(H, yt == MOE_F32 && ot == MOE_F32);
  a.matrix(y, ld_y, yt);
  a.matrix(shared, ld_s, yt);
  a.matrix(out, ld_out, ot);
  with_type(yt, [&](auto* ty) {
    with_type(ot, [&](auto* to) {
      with_n(a.n, [&](auto n) {
        with_waves(tokens, H, a.n, [&](auto w, dim3 grid) {
          using T = std::remove_pointer_t<decltype(ty)>;
          using O = std::remove_pointer_t<decltype(to)>;
          combine_rows<O, T, decltype(n)::value, decltype(w)::value><<<grid, 256, 0, s>>>(
              static_cast<const T*>(y), ld_y, nrows, gates, inv, static_cast<const T*>(shared),
              ld_s, tokens, H, k, static_cast<O*>(out), ld_out);
        });
      });
    });
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_dispatch_workspace_bytes(int64_t tokens, int32_t top_k, int32_t experts) {
  if (check_rows(tokens, 1, top_k) != MOE_OK || experts <= 0 || experts > kMaxExperts) return 0;
  const int64_t TK = tokens * top_k;
  if (TK <= kDispSmall) return 0;
  const int64_t per = chunk_slots(TK);
  return al256((size_t)((TK + per - 1) / per) * experts * sizeof(int32_t));
}

moe_status moe_dispatch(const void* x, int64_t ld_x, moe_dtype dtype, const int32_t* topk_idx,
                        int64_t tokens, int32_t hidden, int32_t top_k, int32_t experts,
                        void* rows, int64_t ld_rows, int32_t* offsets, int32_t* pair,
                        int32_t* inv, void* workspace, size_t workspace_bytes, void* stream) {
  if (!x || !topk_idx || !rows || !offsets || !pair || !inv) return MOE_ERR_NULL;
  const moe_status st = check_rows(tokens, hidden, top_k);
  if (st != MOE_OK) return st;
  if (experts <= 0 || !is_dtype(dtype) || ld_x < hidden || ld_rows < hidden) return MOE_ERR_SHAPE;
  if (experts > kMaxExperts) return MOE_ERR_UNSUPPORTED;
  if (odd_elements(x, dtype) || odd_elements(rows, dtype) || odd4(topk_idx) || odd4(offsets) ||
      odd4(pair) || odd4(inv))
    return MOE_ERR_UNSUPPORTED;
  const size_t need = moe_dispatch_workspace_bytes(tokens, top_k, experts);
  if (need > 0) {
    if (!workspace) return MOE_ERR_NULL;
    if (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
      return MOE_ERR_WORKSPACE;
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t TK = tokens * top_k;
  const int H = hidden, k = top_k, E = experts;
  Shape a(H, dtype == MOE_F32);
  a.matrix(x, ld_x, dtype);
  a.matrix(rows, ld_rows, dtype);
  if (TK <= kDispSmall) {
    with_type(dtype, [&](auto* tp) {
      with_n(a.n, [&](auto n) {
        using T = std::remove_pointer_t<decltype(tp)>;
        constexpr int N = decltype(n)::value;
        const dim3 grid((unsigned)tokens + 1, (unsigned)((H + 256 * N - 1) / (256 * N)));
        dispatch_small<T, N><<<grid, 256, 0, s>>>(static_cast<const T*>(x), ld_x, topk_idx,
                                                  (int)tokens, H, k, E, static_cast<T*>(rows),
                                                  ld_rows, offsets, pair, inv);
      });
    });
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
  }
  const int64_t per = chunk_slots(TK);
  const unsigned chunks = (unsigned)((TK + per - 1) / per);
  int32_t* counts = static_cast<int32_t*>(workspace);
  dispatch_count<<<chunks, 1024, 0, s>>>(topk_idx, TK, per, E, counts);
  dispatch_place<<<chunks, 1024, (size_t)16 * E * sizeof(int32_t), s>>>(topk_idx, TK, per, E,
                                                                        counts, offsets, pair, inv);
  with_type(dtype, [&](auto* tp) {
    with_n(a.n, [&](auto n) {
      with_waves(tokens, H, a.n, [&](auto w, dim3 grid) {
        using T = std::remove_pointer_t<decltype(tp)>;
        dispatch_rows<T, decltype(n)::value, decltype(w)::value><<<grid, 256, 0, s>>>(
            static_cast<const T*>(x), ld_x, tokens, H, k, inv, static_cast<T*>(rows), ld_rows);
      });
    });
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

moe_status moe_dispatch_backward(const void* d_rows, int64_t ld_rows, int64_t rows,
                                 moe_dtype dtype, const int32_t* inv, int64_t tokens,
                                 int32_t hidden, int32_t top_k, void* dx, int64_t ld_dx,
                                 moe_dtype dx_dtype, void* stream) {
  if (!d_rows || !inv || !dx) return MOE_ERR_NULL;
  const moe_status st = check_rows(tokens, hidden, top_k);
  if (st != MOE_OK) return st;
  if (rows < 0 || !is_dtype(dtype) || !is_dtype(dx_dtype) || ld_rows < hidden || ld_dx < hidden)
    return MOE_ERR_SHAPE;
  if (odd_elements(d_rows, dtype) || odd_elements(dx, dx_dtype) || odd4(inv))
    return MOE_ERR_UNSUPPORTED;
  if (tokens == 0) return MOE_OK;
  return launch_combine_rows(d_rows, ld_rows, rows, dtype, nullptr, inv, nullptr, 0, tokens,
                             hidden, top_k, dx, ld_dx, dx_dtype, static_cast<hipStream_t>(stream));
}

moe_status moe_combine(const void* y, int64_t ld_y, int64_t rows, moe_dtype dtype,
                       const float* gates, const int32_t* inv, const void* shared, int64_t ld_shared,
                       int64_t tokens, int32_t hidden, int32_t top_k, void* out, int64_t ld_out,
                       moe_dtype out_dtype, void* stream) {
  if (!y || !gates || !inv || !out) return MOE_ERR_NULL;
  const moe_status st = check_rows(tokens, hidden, top_k);
  if (st != MOE_OK) return st;
  if (rows < 0 || !is_dtype(dtype) || !is_dtype(out_dtype) || ld_y < hidden || ld_out < hidden ||
      (shared && ld_shared < hidden))
    return MOE_ERR_SHAPE;
  if (odd_elements(y, dtype) || odd_elements(shared, dtype) || odd_elements(out, out_dtype) ||
      odd4(gates) || odd4(inv))
    return MOE_ERR_UNSUPPORTED;
  if (tokens == 0) return MOE_OK;
  return launch_combine_rows(y, ld_y, rows, dtype, gates, inv, shared, ld_shared, tokens, hidden,
                             top_k, out, ld_out, out_dtype, static_cast<hipStream_t>(stream));
}

moe_status moe_combine_backward(const void* d_out, int64_t ld_d, moe_dtype d_dtype, const void* y,
                                int64_t ld_y, int64_t rows, moe_dtype dtype, const float* gates,
                                const int32_t* inv, int64_t tokens, int32_t hidden, int32_t top_k,
                                void* d_y, int64_t ld_dy, float* d_gates, void* stream) {
  if (!d_out || !y || !gates || !inv || !d_y || !d_gates) return MOE_ERR_NULL;
  const moe_status st = check_rows(tokens, hidden, top_k);
  if (st != MOE_OK) return st;
  if (rows < 0 || !is_dtype(dtype) || !is_dtype(d_dtype) || ld_y < hidden || ld_d < hidden ||
      ld_dy < hidden)
    return MOE_ERR_SHAPE;
  if (odd_elements(y, dtype) || odd_elements(d_y, dtype) || odd_elements(d_out, d_dtype) ||
      odd4(gates) || odd4(inv) || odd4(d_gates))
    return MOE_ERR_UNSUPPORTED;
  if (tokens == 0) return MOE_OK;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  Shape a(hidden, dtype == MOE_F32 && d_dtype == MOE_F32);
  a.matrix(d_out, ld_d, d_dtype);
  a.matrix(y, ld_y, dtype);
  a.matrix(d_y, ld_dy, dtype);
  const int H = hidden, k = top_k;
  with_type(dtype, [&](auto* ty) {
    with_type(d_dtype, [&](auto* td) {
      with_n(a.n, [&](auto n) {
        using T = std::remove_pointer_t<decltype(ty)>;
        using D = std::remove_pointer_t<decltype(td)>;
        constexpr int N = decltype(n)::value;
        const auto args = [&](auto kernel, unsigned grid) {
          kernel<<<grid, 256, 0, s>>>(static_cast<const D*>(d_out), ld_d, static_cast<const T*>(y),
                                      ld_y, rows, gates, inv, tokens, H, k, static_cast<T*>(d_y),
                                      ld_dy, d_gates);
        };
        if (H <= 64 * N)
          args(combine_grad<D, T, N, 1>, (unsigned)((tokens + 3) / 4));
        else
          args(combine_grad<D, T, N, 4>, (unsigned)tokens);
      });
    });
  });
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

}  // extern "C"
