// Layer normalisation and channel dropout of irreps rows (include/tp_block.h).
//
// Norm.  The blocks of a row are independent, so each is a short row of its own: a CTA works on one
// block of many rows.  A block's floats are read once and kept in registers: its chunks of V floats
// (4, or 2 or 1 where a length or a pointer does not allow 16 or 8 bytes) are dealt to a group of G lanes,
// S chunks a lane, several rows a warp where they are few.  A sum over the block is log2 G shuffles;
// mean first, then the square of what is left of it, both from registers instead of one pass with a
// difference of large sums.  The backward pass keeps every lane's sums of gy n and gy in registers
// over all rows of the lane, adds them up per CTA, and a second kernel adds the CTAs, so gweight and
// gbias cost no extra read of a row and have a fixed order.
//
// Bound by the bytes (8 a float forward, 12 backward) as long as the instructions keep up, which is
// why a block and not a row is the unit: with whole rows a warp (9 chunks a lane at 1,152 floats) the
// sums over three blocks, each chunk asking which one it belongs to, took 365 us for 100,000 rows
// backward, and with whole rows a CTA, through shared memory, 886 us.  8-byte chunks for even lengths:
// 18,262 rows of five blocks of 78 channels went from 78 to 47 us forward and 213 to 102 backward against
// single floats.
//
// Blocks of more than 1,152 floats (36 a lane) take one CTA per row, all blocks of it, with three reads of the
// row, the later ones from L1: k_norm_any.  100,000 rows: 228x2e 147 us forward and 239 backward in registers,
// 256x2e 209 and 903 there.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "../../include/tp_block.h"
#include "philox.cuh"
#include "tp_common.h"
#include "tp_host.h"

namespace tp {
namespace {

constexpr int kNormMaxBlocks = 16;
constexpr int kNormMaxDim = 8192;
constexpr int kNormThreads = 128;

struct NormArgs {
  int64_t N;
  int dim, nb, n_weights, n_bias;
  int off[kNormMaxBlocks], mul[kNormMaxBlocks], d[kNormMaxBlocks];
  int woff[kNormMaxBlocks];     // first weight
  int boff[kNormMaxBlocks];     // first bias, or -1 for a block without a mean
  float inv[kNormMaxBlocks];    // 1 / floats of the block
  int G[kNormMaxBlocks], S[kNormMaxBlocks];     // lanes of a row, chunks a lane
  int cta0[kNormMaxBlocks + 1];                 // first CTA of the block
  float eps;
  const float* x;
  const float* weight;
  const float* bias;
  const float* gy;
  float* y;
  float* gx;
  float* gweight;
  float* gbias;
  // sums over a CTA's rows of gy n and of gy: for each block [its CTAs][2][its floats], from part_at on
  float* part;
  int64_t part_at[kNormMaxBlocks];
};

constexpr int kRowThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

template <int V>
struct Chunk {
  float x[V];
};

template <int V>
__device__ __forceinline__ Chunk<V> read_chunk(const float* p, bool on) {
  Chunk<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.x[i] = 0.0f;
  if (on) {
    if constexpr (V == 4) {
      const float4 t = *reinterpret_cast<const float4*>(p);
      r.x[0] = t.x, r.x[1] = t.y, r.x[2] = t.z, r.x[3] = t.w;
    } else if constexpr (V == 2) {
      const float2 t = *reinterpret_cast<const float2*>(p);
      r.x[0] = t.x, r.x[1] = t.y;
    } else {
      r.x[0] = *p;
    }
  }
  return r;
}

template <int V>
__device__ __forceinline__ void write_chunk(float* p, const Chunk<V>& r) {
  if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(r.x[0], r.x[1], r.x[2], r.x[3]);
  else if constexpr (V == 2) *reinterpret_cast<float2*>(p) = make_float2(r.x[0], r.x[1]);
  else *p = r.x[0];
}

// Weight and bias of every float of block b, in shared memory (a chunk of a block with l > 0 covers parts
// of several channels).
__device__ __forceinline__ void expand_affine(const NormArgs& a, int b, float* w, float* c) {
  const int d = a.d[b], len = a.mul[b] * d;
  for (int i = threadIdx.x; i < len; i += kRowThreads) {
    const int u = i / d;
    w[i] = a.weight ? a.weight[a.woff[b] + u] : 1.0f;
    if (c) c[i] = a.bias && a.boff[b] >= 0 ? a.bias[a.boff[b] + u] : 0.0f;
  }
  __syncthreads();
}

// The lanes of a group and their chunks.
template <int V, int S>
struct RowLanes {
  int G, gl, len;
  float inv, eps;
  bool mean;

  __device__ __forceinline__ RowLanes(const NormArgs& a, int b) {
    G = a.G[b];
    gl = threadIdx.x & (G - 1);
    len = a.mul[b] * a.d[b];
    inv = a.inv[b];
    eps = a.eps;
    mean = a.boff[b] >= 0;
  }
  __device__ __forceinline__ int offset(int s) const { return (s * G + gl) * V; }
  __device__ __forceinline__ bool has(int s) const { return offset(s) < len; }
  __device__ __forceinline__ float sum(float v) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (G > o) v += __shfl_xor_sync(kFull, v, o);
    return v;
  }
  // x becomes n = (x - mu) rho; returns rho.  Chunks that the lane lacks stay 0.
  __device__ __forceinline__ float normalise(Chunk<V> (&x)[S]) const {
    float t = 0.0f;
    if (mean) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) t += x[s].x[i];
      const float mu = sum(t) * inv;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const float m = has(s) ? mu : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) x[s].x[i] -= m;
      }
      t = 0.0f;
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < V; ++i) t = fmaf(x[s].x[i], x[s].x[i], t);
    const float rho = rsqrtf(fmaf(sum(t), inv, eps));
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < V; ++i) x[s].x[i] *= rho;
    return rho;
  }
};

// Rows in flight a group: up to 16 floats a lane on their way, 8 with single floats, whose addresses and
// limits take as many registers as their data (311,042 rows of 21 channels, four blocks, backward: 579 us
// with 8 floats in flight, 622 with 16).  At the registers that ctas_per_sm leaves the backward kernel spills
// some words in the 16- and 8-byte forms too: 60 bytes read back a thread with 16-byte chunks and one a lane, 152
// with 8-byte chunks and up to two.
__host__ __device__ constexpr int rows_in_flight(int V, int S) {
  return V == 4 ? (S == 1 ? 4 : S == 2 ? 2 : 1) : S <= 2 ? 4 : S <= 4 ? 2 : 1;
}

template <int V, int S>
__device__ __forceinline__ void norm_fwd_block(const NormArgs& a, int b, float* affine) {
  constexpr int R = rows_in_flight(V, S);
  const RowLanes<V, S> L(a, b);
  float *w = affine, *c = affine + L.len;
  expand_affine(a, b, w, c);
  const int per = kRowThreads / L.G, mine = threadIdx.x / L.G, cta = blockIdx.x - a.cta0[b], ctas = a.cta0[b + 1] - a.cta0[b];
  const int64_t hop = (int64_t)per * a.dim;
  for (int64_t n0 = (int64_t)cta * per * R + mine; n0 - mine < a.N; n0 += (int64_t)ctas * per * R) {
    Chunk<V> x[R][S];
    const float* xp = a.x + n0 * a.dim + a.off[b];
    float* yp = a.y + n0 * a.dim + a.off[b];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int s = 0; s < S; ++s) x[r][s] = read_chunk<V>(xp + r * hop + L.offset(s), n0 + r * per < a.N && L.has(s));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      L.normalise(x[r]);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (n0 + r * per >= a.N || !L.has(s)) continue;
        const Chunk<V> ws = read_chunk<V>(w + L.offset(s), true), cs = read_chunk<V>(c + L.offset(s), true);
        Chunk<V> y;
#pragma unroll
        for (int i = 0; i < V; ++i) y.x[i] = fmaf(x[r][s].x[i], ws.x[i], cs.x[i]);
        write_chunk<V>(yp + r * hop + L.offset(s), y);
      }
    }
  }
}

// MEAN: a 0e block.
template <int V, int S, bool MEAN>
__device__ __forceinline__ void norm_bwd_block(const NormArgs& a, int b, float* affine) {
  constexpr int R = rows_in_flight(V, S);
  const RowLanes<V, S> L(a, b);
  expand_affine(a, b, affine, nullptr);
  const int per = kRowThreads / L.G, mine = threadIdx.x / L.G, cta = blockIdx.x - a.cta0[b], ctas = a.cta0[b + 1] - a.cta0[b];
  const int64_t hop = (int64_t)per * a.dim;
  Chunk<V> sw[S], sb[S];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < V; ++i) sw[s].x[i] = sb[s].x[i] = 0.0f;
  for (int64_t n0 = (int64_t)cta * per * R + mine; n0 - mine < a.N; n0 += (int64_t)ctas * per * R) {
    Chunk<V> x[R][S], g[R][S];
    const int64_t at = n0 * a.dim + a.off[b];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const bool on = n0 + r * per < a.N && L.has(s);
        x[r][s] = read_chunk<V>(a.x + at + r * hop + L.offset(s), on);
        g[r][s] = read_chunk<V>(a.gy + at + r * hop + L.offset(s), on);
      }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float rho = L.normalise(x[r]);
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) sw[s].x[i] = fmaf(g[r][s].x[i], x[r][s].x[i], sw[s].x[i]);
      if constexpr (MEAN) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) sb[s].x[i] += g[r][s].x[i];
      }
      if (!a.gx) continue;
      float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const Chunk<V> ws = read_chunk<V>(affine + L.offset(s), L.has(s));
#pragma unroll
        for (int i = 0; i < V; ++i) {
          g[r][s].x[i] *= ws.x[i];
          t1 += g[r][s].x[i];
          t2 = fmaf(g[r][s].x[i], x[r][s].x[i], t2);
        }
      }
      t1 = MEAN ? L.sum(t1) * L.inv : 0.0f;
      t2 = L.sum(t2) * L.inv;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (n0 + r * per >= a.N || !L.has(s)) continue;
        Chunk<V> gx;
#pragma unroll
        for (int i = 0; i < V; ++i) gx.x[i] = rho * (g[r][s].x[i] - t1 - x[r][s].x[i] * t2);
        write_chunk<V>(a.gx + at + r * hop + L.offset(s), gx);
      }
    }
  }
  if (!a.part) return;
  // the CTA's sums: lanes of a warp that hold the same chunks by shuffles, then the warps in order
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* sums = affine + warp * 2 * L.len;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o >= L.G) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sw[s].x[i] += __shfl_xor_sync(kFull, sw[s].x[i], o);
          if constexpr (MEAN) sb[s].x[i] += __shfl_xor_sync(kFull, sb[s].x[i], o);
        }
    }
  if (lane < L.G) {
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (L.has(s)) {
        write_chunk<V>(sums + L.offset(s), sw[s]);
        if constexpr (MEAN) write_chunk<V>(sums + L.len + L.offset(s), sb[s]);
      }
  }
  __syncthreads();
  float* out = a.part + a.part_at[b] + (int64_t)cta * 2 * L.len;
  for (int i = threadIdx.x; i < (MEAN ? 2 : 1) * L.len; i += kRowThreads) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowThreads / 32; ++w) t += affine[w * 2 * L.len + i];
    out[i] = t;
  }
}

// CTAs a SM that the registers are held to: a lane keeps three to four arrays of its chunks backward.
__host__ __device__ constexpr int ctas_per_sm(bool bwd, int floats) {
  return bwd ? (floats <= 4 ? 4 : floats <= 8 ? 3 : floats <= 24 ? 2 : 1) : (floats <= 16 ? 4 : floats <= 24 ? 3 : 2);
}

// MOST: the most chunks a lane of any block, which sets the registers; each block runs with its own.
template <bool BWD, int V, int MOST>
__global__ void __launch_bounds__(kRowThreads, ctas_per_sm(BWD, V * MOST)) k_norm(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) float affine[];
  if (BWD) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int b = 0;
  while ((int)blockIdx.x >= a.cta0[b + 1]) ++b;
#define TP_NORM_CASE(n)                                                          \
  case n:                                                                        \
    if constexpr (n <= MOST) {                                                   \
      if constexpr (!BWD) norm_fwd_block<V, n>(a, b, affine);                    \
      else if (a.boff[b] >= 0) norm_bwd_block<V, n, true>(a, b, affine);         \
      else norm_bwd_block<V, n, false>(a, b, affine);                            \
    }                                                                            \
    break;
  if constexpr (V >= 2) {
    switch (a.S[b]) {
      TP_NORM_CASE(1)
      TP_NORM_CASE(2)
      TP_NORM_CASE(3)
      TP_NORM_CASE(4)
      TP_NORM_CASE(6)
      TP_NORM_CASE(9)
      TP_NORM_CASE(18)
    }
  } else {
    switch (a.S[b]) {
      TP_NORM_CASE(1)
      TP_NORM_CASE(2)
      TP_NORM_CASE(4)
      TP_NORM_CASE(8)
      TP_NORM_CASE(16)
      TP_NORM_CASE(24)
      TP_NORM_CASE(36)
    }
  }
#undef TP_NORM_CASE
}

// Sum over the CTA, the same value in every thread.  Two barriers: s is free again afterwards.
__device__ __forceinline__ float cta_sum(float v, float* s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int w = 0; w < kNormThreads / 32; ++w) v += s[w];
  __syncthreads();
  return v;
}

template <bool BWD>
__global__ void __launch_bounds__(kNormThreads) k_norm_any(const __grid_constant__ NormArgs a) {
  extern __shared__ float acc[];          // BWD: [2][dim]
  __shared__ float red[kNormThreads / 32];
  const int tid = threadIdx.x;
  const bool sums = BWD && a.part != nullptr;
  if (sums)
    for (int i = tid; i < 2 * a.dim; i += kNormThreads) acc[i] = 0.0f;
  for (int64_t n = blockIdx.x; n < a.N; n += gridDim.x) {
    const float* x = a.x + n * a.dim;
    for (int b = 0; b < a.nb; ++b) {
      const int len = a.mul[b] * a.d[b], d = a.d[b];
      const float* xb = x + a.off[b];
      const float inv = 1.0f / (float)len;
      float mu = 0.0f;
      if (a.boff[b] >= 0) {
        float t = 0.0f;
        for (int i = tid; i < len; i += kNormThreads) t += xb[i];
        mu = cta_sum(t, red) * inv;
      }
      float t = 0.0f;
      for (int i = tid; i < len; i += kNormThreads) {
        const float c = xb[i] - mu;
        t = fmaf(c, c, t);
      }
      const float rho = rsqrtf(fmaf(cta_sum(t, red), inv, a.eps));
      if (!BWD) {
        float* y = a.y + n * a.dim + a.off[b];
        for (int i = tid; i < len; i += kNormThreads) {
          const int u = i / d;
          const float w = a.weight ? a.weight[a.woff[b] + u] : 1.0f;
          const float c = a.bias && a.boff[b] >= 0 ? a.bias[a.boff[b] + u] : 0.0f;
          y[i] = fmaf((xb[i] - mu) * rho, w, c);
        }
      } else {
        const float* gy = a.gy + n * a.dim + a.off[b];
        float s1 = 0.0f, s2 = 0.0f;
        for (int i = tid; i < len; i += kNormThreads) {
          const float w = a.weight ? a.weight[a.woff[b] + i / d] : 1.0f;
          const float h = (xb[i] - mu) * rho, g = gy[i];
          s1 = fmaf(g, w, s1);
          s2 = fmaf(g * w, h, s2);
          if (sums) {
            acc[a.off[b] + i] = fmaf(g, h, acc[a.off[b] + i]);
            acc[a.dim + a.off[b] + i] += g;
          }
        }
        if (a.gx) {
          s1 = a.boff[b] >= 0 ? cta_sum(s1, red) * inv : 0.0f;
          s2 = cta_sum(s2, red) * inv;
          float* gx = a.gx + n * a.dim + a.off[b];
          for (int i = tid; i < len; i += kNormThreads) {
            const float w = a.weight ? a.weight[a.woff[b] + i / d] : 1.0f;
            const float h = (xb[i] - mu) * rho;
            gx[i] = rho * (gy[i] * w - s1 - h * s2);
          }
        }
      }
    }
  }
  __syncthreads();
  if (sums)
    for (int b = 0; b < a.nb; ++b) {
      const int len = a.mul[b] * a.d[b];
      float* out = a.part + a.part_at[b] + (int64_t)blockIdx.x * 2 * len;
      for (int i = tid; i < len; i += kNormThreads) {
        out[i] = acc[a.off[b] + i];
        out[len + i] = acc[a.dim + a.off[b] + i];
      }
    }
}

// gweight[u] = sum over CTAs and m, gbias[u] = sum over CTAs, in fixed orders.  One CTA for the channels
// that 32 floats of a block hold (32, 10, 6 or 4), a lane a float; its 16 warps take every 16th CTA's
// partials, eight reads in flight each; 64-bit sums, the partials being up to some hundred terms of both
// signs.  With 32 channels a CTA, four CTAs had all the reads of a small row's norm: 14 us for 1,536 rows
// of 288 floats.
constexpr int kSumThreads = 512;

__global__ void __launch_bounds__(kSumThreads) k_norm_sums(const __grid_constant__ NormArgs a) {
  __shared__ double sums[kSumThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int tile = blockIdx.x, b = 0;
  bool bias = false;
  for (;; ++b) {
    if (b == a.nb) {
      bias = true;
      b = 0;
    }
    if (bias && a.boff[b] < 0) continue;
    const int wide = 32 / a.d[b], tiles = (a.mul[b] + wide - 1) / wide;
    if (tile < tiles) break;
    tile -= tiles;
  }
  const int d = a.d[b], wide = 32 / d, u0 = tile * wide, channels = min(wide, a.mul[b] - u0);
  const int len = a.mul[b] * d, ctas = a.cta0[b + 1] - a.cta0[b];
  const float* p = a.part + a.part_at[b] + (bias ? len : 0) + u0 * d + min(lane, channels * d - 1);
  double t = 0.0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll 8
  for (int c = warp; c < ctas; c += kSumThreads / 32) t += (double)p[(int64_t)c * 2 * len];
  sums[warp][lane] = t;
  __syncthreads();
  float* out = bias ? a.gbias : a.gweight;
  if (threadIdx.x < channels && out) {
    double v = 0.0;
    for (int m = 0; m < d; ++m)
#pragma unroll
      for (int w = 0; w < kSumThreads / 32; ++w) v += sums[w][threadIdx.x * d + m];
    out[(bias ? a.boff[b] : a.woff[b]) + u0 + threadIdx.x] = (float)v;
  }
}

// Dropout: a warp takes a row, or several narrow ones, at a time, starts reading
// them, draws the choices of their channels into its part of shared memory meanwhile (one generator
// block for four channels, about 100 instructions) and applies them, G lanes a row.  A table of every
// float's channel, made once a CTA, stands for the divisions.  Bound by the bytes, 8 a float: with tiles of
// rows drawn by a whole CTA between two barriers, a third of the time went to waiting at those (100,000
// rows of 1,152 floats: 193 us).
constexpr int kDropThreads = 256;
constexpr int kDropWarps = kDropThreads / 32;
constexpr int kDropAhead = 6;          // chunks of a lane in flight

struct DropoutArgs {
  int64_t N;
  int dim, C, nb, tile, G;             // rows a warp takes, lanes per row
  int off[kNormMaxBlocks], d[kNormMaxBlocks], coff[kNormMaxBlocks];
  const float* x;
  float* y;
  DropArgs drop;
};

size_t drop_chan_bytes(int dim) { return (2 * (size_t)dim + 15) & ~(size_t)15; }
__host__ __device__ inline int drop_words(int tile, int C) { return (tile * C + 3) / 4 + 1; }

template <int V>
__global__ void __launch_bounds__(kDropThreads) k_dropout(const __grid_constant__ DropoutArgs a) {
  extern __shared__ __align__(16) unsigned char sm[];
  uint16_t* chan = reinterpret_cast<uint16_t*>(sm);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // keep bytes, four a word
  uint32_t* words = reinterpret_cast<uint32_t*>(sm + ((2 * (size_t)a.dim + 15) & ~(size_t)15)) + warp * drop_words(a.tile, a.C);
  for (int i = threadIdx.x; i < a.dim; i += kDropThreads) {
    int b = a.nb - 1;
    while (b > 0 && i < a.off[b]) --b;
    chan[i] = (uint16_t)(a.coff[b] + (i - a.off[b]) / a.d[b]);
  }
  const DropKey key = drop_key(a.drop);
  __syncthreads();
  const int chunks = a.dim / V, gl = lane & (a.G - 1), group = lane / a.G, groups = 32 / a.G;
  const bool narrow = chunks <= a.G;     // a lane's chunks in flight are those of several rows, not of one
  const int64_t warps = (int64_t)gridDim.x * kDropWarps;
  for (int64_t t = (int64_t)blockIdx.x * kDropWarps + warp; t * a.tile < a.N; t += warps) {
    const int64_t row0 = t * a.tile;
    const int rows = (int)min((int64_t)a.tile, a.N - row0);
    const float* x = a.x + row0 * a.dim;
    float* y = a.y + row0 * a.dim;
    bool drawn = false;
    const uint64_t first = (uint64_t)row0 * a.C;
    const int shift = (int)(first & 3), blocks = (rows * a.C + shift + 3) / 4;
    for (int r0 = 0; r0 < rows; r0 += groups * (narrow ? kDropAhead : 1)) {
      for (int c0 = gl; c0 - gl < chunks; c0 += kDropAhead * a.G) {
        Chunk<V> v[kDropAhead];
#pragma unroll
        for (int i = 0; i < kDropAhead; ++i) {
          const int r = r0 + group + (narrow ? i * groups : 0), c = c0 + (narrow ? 0 : i * a.G);
          v[i] = read_chunk<V>(x + (int64_t)r * a.dim + c * V, r < rows && c < chunks);
        }
        if (!drawn) {
          drawn = true;
          __syncwarp();
          for (int i = lane; i < blocks; i += 32) words[i] = keep_bytes(key, a.drop.threshold, (first >> 2) + i);
          __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < kDropAhead; ++i) {
          const int r = r0 + group + (narrow ? i * groups : 0), c = c0 + (narrow ? 0 : i * a.G);
          if (r >= rows || c >= chunks) break;
          const unsigned char* keep = reinterpret_cast<const unsigned char*>(words) + shift + r * a.C;
          if constexpr (V == 4) {
            const ushort4 u = *reinterpret_cast<const ushort4*>(chan + 4 * c);
            v[i].x[0] = keep[u.x] ? v[i].x[0] * a.drop.inv_keep : 0.0f;
            v[i].x[1] = keep[u.y] ? v[i].x[1] * a.drop.inv_keep : 0.0f;
            v[i].x[2] = keep[u.z] ? v[i].x[2] * a.drop.inv_keep : 0.0f;
            v[i].x[3] = keep[u.w] ? v[i].x[3] * a.drop.inv_keep : 0.0f;
          } else {
            v[i].x[0] = keep[chan[c]] ? v[i].x[0] * a.drop.inv_keep : 0.0f;
          }
          write_chunk<V>(y + (int64_t)r * a.dim + c * V, v[i]);
        }
      }
    }
  }
}

bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
tp_status_t cuda_status(cudaError_t e, const char* where) {
  return e == cudaSuccess ? TP_OK : set_failure(TP_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

// Parses an irreps string and checks the limits both operators share.
tp_status_t parse_rows(const char* irreps, std::vector<IrrepTerm>& t, int& dim) {
  std::string why;
  if (!parse_irreps_terms(irreps, t, why)) return set_failure(TP_ERR_INVALID_ARG, "irreps: " + why);
  if ((int)t.size() > kNormMaxBlocks) return set_failure(TP_ERR_UNSUPPORTED, "at most 16 irreps blocks");
  int64_t n = 0;
  for (const IrrepTerm& b : t) {
    if (b.l > 3) return set_failure(TP_ERR_UNSUPPORTED, "l > 3");
    n += (int64_t)b.mul * (2 * b.l + 1);
  }
  if (n > kNormMaxDim) return set_failure(TP_ERR_UNSUPPORTED, "rows of at most 8192 floats");
  dim = (int)n;
  return TP_OK;
}

// Lanes and chunks a lane of each block: the fewest idle lanes among the forms with at most sixteen floats a
// lane, and of those with equally few the one with most lanes; a whole warp for longer blocks.  Returns the
// most chunks a lane, 0 if a block is too long.
int row_forms(NormArgs& a, int V) {
  static const int slots4[] = {1, 2, 3, 4, 6, 9, 18}, slots1[] = {1, 2, 4, 8, 16, 24, 36};
  int most = 0;
  for (int b = 0; b < a.nb; ++b) {
    const int chunks = a.mul[b] * a.d[b] / V;
    a.S[b] = 0;
    for (int G = 32; G >= 1; G /= 2) {
      int S = 0;
      if (V >= 2) {
        for (int s : slots4)
          if (S == 0 && s * G >= chunks && V * s <= 36) S = s;
      } else {
        for (int s : slots1)
          if (S == 0 && s * G >= chunks) S = s;
      }
      if (S == 0 || (a.S[b] != 0 && (S * V > 16 || G * S >= a.G[b] * a.S[b]))) continue;
      a.G[b] = G;
      a.S[b] = S;
    }
    if (a.S[b] == 0) return 0;
    most = std::max(most, a.S[b]);
  }
  return most;
}

// Shares `total` CTAs out among the blocks by their floats, at least one each and none without a row.
// `any`: one row a CTA and every CTA on all blocks (k_norm_any).
void share_ctas(NormArgs& a, int64_t N, int total, int V, bool any) {
  int64_t at = 0;
  a.cta0[0] = 0;
  for (int b = 0; b < a.nb; ++b) {
    const int len = a.mul[b] * a.d[b];
    int64_t n;
    if (any) {
      n = std::min<int64_t>(N, total);
    } else {
      const int per = kRowThreads / a.G[b] * rows_in_flight(V, a.S[b]);
      n = std::min<int64_t>((N + per - 1) / per, ((int64_t)total * len + a.dim - 1) / a.dim);
    }
    n = std::max<int64_t>(n, 1);
    a.cta0[b + 1] = a.cta0[b] + (int)n;
    a.part_at[b] = at;
    at += n * 2 * len;
  }
}

// CTAs of the backward pass: what is resident at once, each leaves a partial of the weight gradients.
int most_slots(int most, int V) {
  if (V == 4) return most <= 1 ? 1 : most <= 2 ? 2 : most <= 4 ? 4 : most <= 6 ? 6 : 9;
  if (V == 2) return most <= 2 ? 2 : most <= 4 ? 4 : most <= 9 ? 9 : 18;
  return most <= 4 ? 4 : most <= 8 ? 8 : most <= 16 ? 16 : 36;
}
int bwd_ctas(const NormArgs& a, int most, int V) {
  if (most == 0) return 148 * std::max(1, std::min(8, 160 * 1024 / (8 * a.dim)));
  return 148 * ctas_per_sm(true, V * most_slots(most, V));
}

// Floats of the partials with any width of a chunk up to `width`: the workspace does not depend on alignment.
size_t part_floats(const NormArgs& proto, int width, int64_t N) {
  size_t n = 0;
  for (int V : {1, 2, 4}) {
    if (V > width) continue;
    NormArgs a = proto;
    const int most = row_forms(a, V);
    share_ctas(a, N, bwd_ctas(a, most, V), V, most == 0);
    const int b = a.nb - 1;
    n = std::max(n, (size_t)a.part_at[b] + (size_t)(a.cta0[b + 1] - a.cta0[b]) * 2 * a.mul[b] * a.d[b]);
  }
  return n;
}

template <bool BWD, int V, int MOST>
cudaError_t launch_most(const NormArgs& a, size_t smem, cudaStream_t s) {
  if (smem > 40 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(k_norm<BWD, V, MOST>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  k_norm<BWD, V, MOST><<<a.cta0[a.nb], kRowThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <bool BWD>
cudaError_t launch_norm(const NormArgs& a, int most, int V, cudaStream_t s) {
  int len = 0;
  for (int b = 0; b < a.nb; ++b) len = std::max(len, a.mul[b] * a.d[b]);
  const size_t smem = sizeof(float) * 2 * (size_t)len * (BWD && a.part ? kRowThreads / 32 : 1);
  switch (most_slots(most, V) * 8 + V) {
    case 1 * 8 + 4: return launch_most<BWD, 4, 1>(a, smem, s);
    case 2 * 8 + 4: return launch_most<BWD, 4, 2>(a, smem, s);
    case 4 * 8 + 4: return launch_most<BWD, 4, 4>(a, smem, s);
    case 6 * 8 + 4: return launch_most<BWD, 4, 6>(a, smem, s);
    case 9 * 8 + 4: return launch_most<BWD, 4, 9>(a, smem, s);
    case 2 * 8 + 2: return launch_most<BWD, 2, 2>(a, smem, s);
    case 4 * 8 + 2: return launch_most<BWD, 2, 4>(a, smem, s);
    case 9 * 8 + 2: return launch_most<BWD, 2, 9>(a, smem, s);
    case 18 * 8 + 2: return launch_most<BWD, 2, 18>(a, smem, s);
    case 4 * 8 + 1: return launch_most<BWD, 1, 4>(a, smem, s);
    case 8 * 8 + 1: return launch_most<BWD, 1, 8>(a, smem, s);
    case 16 * 8 + 1: return launch_most<BWD, 1, 16>(a, smem, s);
    default: return launch_most<BWD, 1, 36>(a, smem, s);
  }
}

// The widest chunk, up to `width` floats, that the pointers allow.
int chunk_width(int width, const void* p, const void* q, const void* r) {
  for (const void* t : {p, q, r})
    while (reinterpret_cast<uintptr_t>(t) % (4 * width) != 0) width /= 2;
  return width;
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace tp

using namespace tp;

struct tp_norm_s {
  NormArgs proto;
  int width;                 // the largest of 4, 2, 1 that divides every block's length
};
struct tp_dropout_s {
  DropoutArgs proto;
};

extern "C" {

tp_status_t tp_norm_create(tp_norm_t* norm, const char* irreps, double eps) try {
  if (!norm) return set_failure(TP_ERR_INVALID_ARG, "norm is NULL");
  *norm = nullptr;
  std::vector<IrrepTerm> t;
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  tp_status_t st = parse_rows(irreps, t, a.dim);
  if (st != TP_OK) return st;
  // squares below 2^-126 are flushed to zero, at most 2^-26 of such an eps
  if (!((float)eps >= 1.0e-30f && (float)eps <= 3.0e38f)) return set_failure(TP_ERR_INVALID_ARG, "eps must be at least 1e-30 and finite");
  a.eps = (float)eps;
  int off = 0;
  int width = 4;
  for (const IrrepTerm& b : t) {
    const int i = a.nb++;
    while (b.mul * (2 * b.l + 1) % width != 0) width /= 2;
    a.off[i] = off;
    a.mul[i] = b.mul;
    a.d[i] = 2 * b.l + 1;
    a.inv[i] = 1.0f / (float)(a.mul[i] * a.d[i]);
    a.woff[i] = a.n_weights;
    a.boff[i] = -1;
    if (b.l == 0 && b.parity == 1) {
      a.boff[i] = a.n_bias;
      a.n_bias += b.mul;
    }
    a.n_weights += b.mul;
    off += b.mul * a.d[i];
  }
  tp_norm_s* h = new tp_norm_s();
  h->proto = a;
  h->width = width;
  *norm = h;
  return TP_OK;
} catch (...) {
  return TP_ERR_INVALID_ARG;   // out of host memory
}

tp_status_t tp_norm_destroy(tp_norm_t norm) {
  delete norm;
  return TP_OK;
}

tp_status_t tp_norm_query(tp_norm_t norm, int64_t* dim, int64_t* n_weights, int64_t* n_bias) {
  if (!norm) return set_failure(TP_ERR_INVALID_ARG, "norm is NULL");
  if (dim) *dim = norm->proto.dim;
  if (n_weights) *n_weights = norm->proto.n_weights;
  if (n_bias) *n_bias = norm->proto.n_bias;
  return TP_OK;
}

tp_status_t tp_norm_workspace_size(tp_norm_t norm, int64_t N, int32_t op, size_t* bytes) {
  if (!norm || !bytes) return set_failure(TP_ERR_INVALID_ARG, "NULL argument");
  if (N < 0) return set_failure(TP_ERR_INVALID_ARG, "N must be non-negative");
  if (op != TP_OP_FWD && op != TP_OP_BWD) return set_failure(TP_ERR_INVALID_ARG, "op must be TP_OP_FWD or TP_OP_BWD");
  *bytes = op == TP_OP_FWD ? 0 : sizeof(float) * part_floats(norm->proto, norm->width, N);
  return TP_OK;
}

tp_status_t tp_norm_fwd(tp_norm_t norm, int64_t N, const float* x, const float* weight, const float* bias, float* y,
                        tp_stream_t stream) {
  if (!norm) return set_failure(TP_ERR_INVALID_ARG, "norm is NULL");
  if (N < 0) return set_failure(TP_ERR_INVALID_ARG, "N must be non-negative");
  if (N >= (int64_t)1 << 40) return set_failure(TP_ERR_UNSUPPORTED, "N too large");
  if (N == 0) return TP_OK;
  if (!x || !y) return set_failure(TP_ERR_INVALID_ARG, "x and y must not be NULL");
  if (!al4(x) || !al4(weight) || !al4(bias) || !al4(y))
    return set_failure(TP_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  NormArgs a = norm->proto;
  a.N = N;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int V = chunk_width(norm->width, x, y, nullptr), most = row_forms(a, V);
  count_launches(1);
  if (most == 0) {
    k_norm_any<false><<<(unsigned)std::min<int64_t>(N, 148 * 16), kNormThreads, 0, s>>>(a);
    return cuda_status(cudaGetLastError(), "tp_norm_fwd");
  }
  share_ctas(a, N, 148 * 8, V, false);
  return cuda_status(launch_norm<false>(a, most, V, s), "tp_norm_fwd");
}

tp_status_t tp_norm_bwd(tp_norm_t norm, int64_t N, const float* x, const float* weight, const float* gy, float* gx,
                        float* gweight, float* gbias, void* ws, size_t ws_bytes, tp_stream_t stream) {
  if (!norm) return set_failure(TP_ERR_INVALID_ARG, "norm is NULL");
  if (N < 0) return set_failure(TP_ERR_INVALID_ARG, "N must be non-negative");
  if (N >= (int64_t)1 << 40) return set_failure(TP_ERR_UNSUPPORTED, "N too large");
  const bool sums = gweight || (gbias && norm->proto.n_bias > 0);
  if (!sums && (!gx || N == 0)) return TP_OK;
  if (N > 0 && (!x || !gy)) return set_failure(TP_ERR_INVALID_ARG, "x and gy must not be NULL");
  if (!al4(x) || !al4(weight) || !al4(gy) || !al4(gx) || !al4(gweight) || !al4(gbias) || !al4(ws))
    return set_failure(TP_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  NormArgs a = norm->proto;
  a.N = N;
  a.x = x;
  a.weight = weight;
  a.gy = gy;
  a.gx = gx;
  a.gweight = gweight;
  a.gbias = gbias;
  const size_t need = sums ? sizeof(float) * part_floats(a, norm->width, N) : 0;
  if (sums && (!ws || ws_bytes < need)) return set_failure(TP_ERR_WORKSPACE, "workspace too small");
  a.part = sums ? static_cast<float*>(ws) : nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int V = chunk_width(norm->width, x, gy, gx), most = row_forms(a, V);
  share_ctas(a, N, bwd_ctas(a, most, V), V, most == 0);
  cudaError_t e = cudaSuccess;
  count_launches(1);
  if (most == 0) {
    const int smem = sums ? (int)(sizeof(float) * 2 * a.dim) : 0;
    if (smem > 40 * 1024) e = cudaFuncSetAttribute(k_norm_any<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_status(e, "tp_norm_bwd");
    k_norm_any<true><<<a.cta0[1], kNormThreads, smem, s>>>(a);
    e = cudaGetLastError();
  } else {
    e = launch_norm<true>(a, most, V, s);
  }
  if (e == cudaSuccess && sums) {
    unsigned tiles = 0;
    for (int b = 0; b < a.nb; ++b) {
      const int wide = 32 / a.d[b];
      tiles += (unsigned)((a.mul[b] + wide - 1) / wide) * (a.boff[b] >= 0 ? 2 : 1);
    }
    cudaLaunchAttribute attr;            // set up while the first kernel runs; it waits for its end
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(tiles);
    c.blockDim = dim3(kSumThreads);
    c.stream = s;
    c.attrs = &attr;
    c.numAttrs = 1;
    count_launches(1);
    e = cudaLaunchKernelEx(&c, k_norm_sums, a);
  }
  return cuda_status(e, "tp_norm_bwd");
}

tp_status_t tp_dropout_create(tp_dropout_t* drop, const char* irreps) try {
  if (!drop) return set_failure(TP_ERR_INVALID_ARG, "dropout is NULL");
  *drop = nullptr;
  std::vector<IrrepTerm> t;
  DropoutArgs a;
  std::memset(&a, 0, sizeof(a));
  tp_status_t st = parse_rows(irreps, t, a.dim);
  if (st != TP_OK) return st;
  int off = 0;
  for (const IrrepTerm& b : t) {
    a.off[a.nb] = off;
    a.d[a.nb] = 2 * b.l + 1;
    a.coff[a.nb] = a.C;
    a.C += b.mul;
    off += b.mul * a.d[a.nb++];
  }
  tp_dropout_s* h = new tp_dropout_s();
  h->proto = a;
  *drop = h;
  return TP_OK;
} catch (...) {
  return TP_ERR_INVALID_ARG;   // out of host memory
}

tp_status_t tp_dropout_destroy(tp_dropout_t drop) {
  delete drop;
  return TP_OK;
}

tp_status_t tp_dropout_query(tp_dropout_t drop, int64_t* dim, int64_t* n_channels) {
  if (!drop) return set_failure(TP_ERR_INVALID_ARG, "dropout is NULL");
  if (dim) *dim = drop->proto.dim;
  if (n_channels) *n_channels = drop->proto.C;
  return TP_OK;
}

tp_status_t tp_dropout_fwd(tp_dropout_t drop, int64_t N, const float* x, double p, const int64_t* rng, int64_t site,
                           float* y, tp_stream_t stream) {
  if (!drop) return set_failure(TP_ERR_INVALID_ARG, "dropout is NULL");
  if (N < 0) return set_failure(TP_ERR_INVALID_ARG, "N must be non-negative");
  if (N >= (int64_t)1 << 40) return set_failure(TP_ERR_UNSUPPORTED, "N too large");
  DropoutArgs a = drop->proto;
  if (!drop_args(p, rng, site, a.drop))
    return set_failure(TP_ERR_INVALID_ARG, "p must lie in [0, 1) and p > 0 needs rng");
  if (N == 0) return TP_OK;
  if (!x || !y) return set_failure(TP_ERR_INVALID_ARG, "input and output must not be NULL");
  if (!al4(x) || !al4(y) || (reinterpret_cast<uintptr_t>(rng) & 7u))
    return set_failure(TP_ERR_INVALID_ARG, "pointers must be 4-byte aligned, rng 8-byte aligned");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!a.drop.rng) {
    if (x == y) return TP_OK;
    return cuda_status(cudaMemcpyAsync(y, x, sizeof(float) * (size_t)N * a.dim, cudaMemcpyDeviceToDevice, s), "tp_dropout");
  }
  a.N = N;
  a.x = x;
  a.y = y;
  const bool vec4 = a.dim % 4 == 0 && al16(x) && al16(y);
  const int chunks = vec4 ? a.dim / 4 : a.dim;
  a.G = 1;
  while (a.G < 32 && a.G < chunks) a.G *= 2;
  // one long row, or rows that give every lane its chunks in flight, and fewer where warps would have none
  a.tile = chunks > a.G ? 1 : 32 / a.G * kDropAhead;
  a.tile = (int)std::max<int64_t>(std::min<int64_t>(a.tile, N / (148 * 16)), 1);
  const size_t smem = drop_chan_bytes(a.dim) + 4 * (size_t)kDropWarps * drop_words(a.tile, a.C);
  const int64_t tiles = (N + (int64_t)a.tile * kDropWarps - 1) / ((int64_t)a.tile * kDropWarps);
  const unsigned grid = (unsigned)std::min<int64_t>(tiles, 148 * 8);
  auto kernel = vec4 ? k_dropout<4> : k_dropout<1>;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return cuda_status(e, "tp_dropout");
  }
  kernel<<<grid, kDropThreads, smem, s>>>(a);
  count_launches(1);
  return cuda_status(cudaGetLastError(), "tp_dropout");
}

tp_status_t tp_dropout_bwd(tp_dropout_t drop, int64_t N, const float* gy, double p, const int64_t* rng, int64_t site,
                           float* gx, tp_stream_t stream) {
  return tp_dropout_fwd(drop, N, gy, p, rng, site, gx, stream);
}

}  // extern "C"
