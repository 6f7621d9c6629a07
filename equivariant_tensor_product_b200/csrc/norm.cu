// Layer normalisation and channel dropout of irreps rows (include/tp_block.h).
//
// Norm.  A row is read once and kept in registers: its chunks of V floats (4, or 1 where a block's
// length or a pointer does not allow 16 bytes) are dealt to a group of G lanes, S chunks a lane --
// several rows a warp for narrow rows, a warp a row up to 9 chunks a lane, a CTA a row beyond.  A
// chunk lies in one block, so a block's sum is the lanes' sums over their chunks of that block,
// joined by shuffles: mean first, then the square of what is left of it, both in two reads of
// registers instead of one pass with a difference of large sums.  Bound by the bytes (8 a float
// forward, 12 backward).  The backward pass keeps every lane's sums of gy n and gy in registers over
// all rows of the lane, adds them up per CTA, and a second kernel adds the CTAs, so gweight and
// gbias cost no extra read of a row and have a fixed order.
//
// Rows that fit neither form (more than 2,048 chunks) take one CTA per row with three reads of the
// row, the later ones from L1: k_norm_any.
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
constexpr int kNormMaxCtas = 148 * 2;

struct NormArgs {
  int64_t N;
  int dim, nb, n_weights, n_bias;
  int off[kNormMaxBlocks], mul[kNormMaxBlocks], d[kNormMaxBlocks];
  int woff[kNormMaxBlocks];     // first weight
  int boff[kNormMaxBlocks];     // first bias, or -1 for a block without a mean
  float eps;
  const float* x;
  const float* weight;
  const float* bias;
  const float* gy;
  float* y;
  float* gx;
  float* gweight;
  float* gbias;
  float* part;                  // [ctas][2][dim]: sums over a CTA's rows of gy n and of gy
  int ctas;
  int G;                        // lanes of a row (one CTA a row: all its threads)
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
    } else {
      r.x[0] = *p;
    }
  }
  return r;
}

template <int V>
__device__ __forceinline__ void write_chunk(float* p, const Chunk<V>& r) {
  if constexpr (V == 4) *reinterpret_cast<float4*>(p) = make_float4(r.x[0], r.x[1], r.x[2], r.x[3]);
  else *p = r.x[0];
}

// The lanes of a row and the block of each of a lane's chunks.
template <int V, int S, bool CTA>
struct RowLanes {
  int G, gl, bid[S];
  float* red;                // CTA: [2][kRowThreads / 32], used in turn
  int turn;

  __device__ __forceinline__ RowLanes(const NormArgs& a, float* shared) : red(shared), turn(0) {
    G = CTA ? kRowThreads : a.G;
    gl = CTA ? threadIdx.x : threadIdx.x & (a.G - 1);
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int at = offset(s);
      int b = a.nb - 1;
      while (b > 0 && at < a.off[b]) --b;
      bid[s] = at < a.dim ? b : -1;
    }
  }
  __device__ __forceinline__ int offset(int s) const { return (s * G + gl) * V; }
  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (CTA || G > o) v += __shfl_xor_sync(kFull, v, o);
    if constexpr (CTA) {
      float* r = red + turn * (kRowThreads / 32);
      turn ^= 1;
      if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
      __syncthreads();
      v = 0.0f;
#pragma unroll
      for (int w = 0; w < kRowThreads / 32; ++w) v += r[w];
    }
    return v;
  }
  // x becomes n = (x - mu) rho; rho of each chunk's block.
  __device__ __forceinline__ void normalise(const NormArgs& a, Chunk<V> (&x)[S], float (&rho)[S]) {
    for (int b = 0; b < a.nb; ++b) {
      const float inv = 1.0f / (float)(a.mul[b] * a.d[b]);
      float t = 0.0f;
      if (a.boff[b] >= 0) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) t += bid[s] == b ? x[s].x[i] : 0.0f;
        const float mu = sum(t) * inv;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) x[s].x[i] -= bid[s] == b ? mu : 0.0f;
      }
      t = 0.0f;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) q = fmaf(x[s].x[i], x[s].x[i], q);
        t += bid[s] == b ? q : 0.0f;
      }
      const float r = rsqrtf(fmaf(sum(t), inv, a.eps));
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (bid[s] == b) rho[s] = r;
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < V; ++i) x[s].x[i] *= rho[s];
  }
};

// Weight and bias of every float of a row, in shared memory (a chunk of a block with l > 0 covers parts of
// several channels).
__device__ __forceinline__ void expand_affine(const NormArgs& a, float* w, float* c) {
  for (int i = threadIdx.x; i < a.dim; i += kRowThreads) {
    int b = a.nb - 1;
    while (b > 0 && i < a.off[b]) --b;
    const int u = (i - a.off[b]) / a.d[b];
    w[i] = a.weight ? a.weight[a.woff[b] + u] : 1.0f;
    if (c) c[i] = a.bias && a.boff[b] >= 0 ? a.bias[a.boff[b] + u] : 0.0f;
  }
  __syncthreads();
}

template <int V, int S, int R, bool CTA>
__global__ void __launch_bounds__(kRowThreads) k_norm_fwd(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) float affine[];
  __shared__ float red[2 * (kRowThreads / 32)];
  float *w = affine, *c = affine + a.dim;
  expand_affine(a, w, c);
  RowLanes<V, S, CTA> L(a, red);
  const int per = CTA ? 1 : kRowThreads / L.G, mine = CTA ? 0 : threadIdx.x / L.G;
  for (int64_t n0 = (int64_t)blockIdx.x * per * R; n0 < a.N; n0 += (int64_t)gridDim.x * per * R) {
    Chunk<V> x[R][S];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t n = n0 + (int64_t)r * per + mine;
#pragma unroll
      for (int s = 0; s < S; ++s) x[r][s] = read_chunk<V>(a.x + n * a.dim + L.offset(s), n < a.N && L.bid[s] >= 0);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t n = n0 + (int64_t)r * per + mine;
      float rho[S] = {};
      L.normalise(a, x[r], rho);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (n >= a.N || L.bid[s] < 0) continue;
        const Chunk<V> ws = read_chunk<V>(w + L.offset(s), true), cs = read_chunk<V>(c + L.offset(s), true);
        Chunk<V> y;
#pragma unroll
        for (int i = 0; i < V; ++i) y.x[i] = fmaf(x[r][s].x[i], ws.x[i], cs.x[i]);
        write_chunk<V>(a.y + n * a.dim + L.offset(s), y);
      }
    }
  }
}

template <int V, int S, int R, bool CTA>
__global__ void __launch_bounds__(kRowThreads) k_norm_bwd(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) float affine[];
  __shared__ float red[2 * (kRowThreads / 32)];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  float* w = affine;
  expand_affine(a, w, nullptr);
  RowLanes<V, S, CTA> L(a, red);
  const int per = CTA ? 1 : kRowThreads / L.G, mine = CTA ? 0 : threadIdx.x / L.G;
  Chunk<V> sw[S], sb[S];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < V; ++i) sw[s].x[i] = sb[s].x[i] = 0.0f;
  for (int64_t n0 = (int64_t)blockIdx.x * per * R; n0 < a.N; n0 += (int64_t)gridDim.x * per * R) {
    Chunk<V> x[R][S], g[R][S];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t n = n0 + (int64_t)r * per + mine;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const bool on = n < a.N && L.bid[s] >= 0;
        x[r][s] = read_chunk<V>(a.x + n * a.dim + L.offset(s), on);
        g[r][s] = read_chunk<V>(a.gy + n * a.dim + L.offset(s), on);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t n = n0 + (int64_t)r * per + mine;
      float rho[S] = {};
      L.normalise(a, x[r], rho);
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sw[s].x[i] = fmaf(g[r][s].x[i], x[r][s].x[i], sw[s].x[i]);
          sb[s].x[i] += g[r][s].x[i];
        }
      if (!a.gx) continue;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const Chunk<V> ws = read_chunk<V>(w + L.offset(s), L.bid[s] >= 0);
#pragma unroll
        for (int i = 0; i < V; ++i) g[r][s].x[i] *= ws.x[i];
      }
      float s1[S] = {}, s2[S] = {};
      for (int b = 0; b < a.nb; ++b) {
        const float inv = 1.0f / (float)(a.mul[b] * a.d[b]);
        float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          float u1 = 0.0f, u2 = 0.0f;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            u1 += g[r][s].x[i];
            u2 = fmaf(g[r][s].x[i], x[r][s].x[i], u2);
          }
          t1 += L.bid[s] == b ? u1 : 0.0f;
          t2 += L.bid[s] == b ? u2 : 0.0f;
        }
        t1 = a.boff[b] >= 0 ? L.sum(t1) * inv : 0.0f;
        t2 = L.sum(t2) * inv;
#pragma unroll
        for (int s = 0; s < S; ++s)
          if (L.bid[s] == b) {
            s1[s] = t1;
            s2[s] = t2;
          }
      }
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (n >= a.N || L.bid[s] < 0) continue;
        Chunk<V> gx;
#pragma unroll
        for (int i = 0; i < V; ++i) gx.x[i] = rho[s] * (g[r][s].x[i] - s1[s] - x[r][s].x[i] * s2[s]);
        write_chunk<V>(a.gx + n * a.dim + L.offset(s), gx);
      }
    }
  }
  if (!a.part) return;
  // the CTA's sums: lanes of a warp that hold the same chunks, then warp after warp
  float* total = affine;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.dim; i += kRowThreads) total[i] = 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (!CTA && o >= L.G) {
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          sw[s].x[i] += __shfl_xor_sync(kFull, sw[s].x[i], o);
          sb[s].x[i] += __shfl_xor_sync(kFull, sb[s].x[i], o);
        }
    }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int turn = 0; turn < (CTA ? 1 : kRowThreads / 32); ++turn) {
    if (CTA || (warp == turn && lane < L.G)) {
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (L.bid[s] >= 0) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            total[L.offset(s) + i] += sw[s].x[i];
            total[a.dim + L.offset(s) + i] += sb[s].x[i];
          }
        }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < 2 * a.dim; i += kRowThreads) a.part[(int64_t)blockIdx.x * 2 * a.dim + i] = total[i];
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
    for (int i = tid; i < 2 * a.dim; i += kNormThreads) a.part[(int64_t)blockIdx.x * 2 * a.dim + i] = acc[i];
}

// gweight[u] = sum over CTAs and m, gbias[u] = sum over CTAs, in fixed orders.  One CTA for 32 channels of
// a block: its warps take every 16th CTA's partials, whose floats they read side by side; 64-bit sums,
// the partials being up to a few hundred terms of both signs.
constexpr int kSumThreads = 512;

__global__ void __launch_bounds__(kSumThreads) k_norm_sums(const __grid_constant__ NormArgs a) {
  __shared__ double sums[kSumThreads / 32][7 * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int tile = blockIdx.x, b = 0;
  bool bias = false;
  for (;; ++b) {
    if (b == a.nb) {
      bias = true;
      b = 0;
    }
    if (bias && a.boff[b] < 0) continue;
    const int tiles = (a.mul[b] + 31) / 32;
    if (tile < tiles) break;
    tile -= tiles;
  }
  const int d = bias ? 1 : a.d[b], u0 = tile * 32, channels = min(32, a.mul[b] - u0);
  const float* p = a.part + (bias ? a.dim : 0) + a.off[b] + u0 * d;
  double t[7] = {};
  asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll 4
  for (int c = warp; c < a.ctas; c += kSumThreads / 32) {
#pragma unroll
    for (int m = 0; m < 7; ++m) {
      const int i = m * 32 + lane;
      if (m < d && i < channels * d) t[m] += (double)p[(int64_t)c * 2 * a.dim + i];
    }
  }
#pragma unroll
  for (int m = 0; m < 7; ++m) sums[warp][m * 32 + lane] = t[m];
  __syncthreads();
  float* out = bias ? a.gbias : a.gweight;
  if (threadIdx.x < channels && out) {
    double v = 0.0;
    for (int m = 0; m < d; ++m)
      for (int w = 0; w < kSumThreads / 32; ++w) v += sums[w][threadIdx.x * d + m];
    out[(bias ? a.boff[b] : a.woff[b]) + u0 + threadIdx.x] = (float)v;
  }
}

// Dropout: a CTA takes a tile of consecutive rows, draws the choices of their channels into
// shared memory (one generator block for four channels, about 100 instructions) and then passes
// over the tile's floats, G lanes a row, up to four chunks of a lane in flight.  A table of every
// float's channel, made once a CTA, stands for the divisions.  Bound by the bytes, 8 a float.
constexpr int kDropThreads = 256;
constexpr int kDropMaxWords = 4096;    // channels of a tile

struct DropoutArgs {
  int64_t N;
  int dim, C, nb, tile, G;             // rows per tile, lanes per row
  int off[kNormMaxBlocks], d[kNormMaxBlocks], coff[kNormMaxBlocks];
  const float* x;
  float* y;
  DropArgs drop;
};

template <int V>
__global__ void __launch_bounds__(kDropThreads) k_dropout(const __grid_constant__ DropoutArgs a) {
  extern __shared__ __align__(16) unsigned char sm[];
  uint16_t* chan = reinterpret_cast<uint16_t*>(sm);
  uint32_t* words = reinterpret_cast<uint32_t*>(sm + ((2 * (size_t)a.dim + 15) & ~(size_t)15));   // keep bytes, four a word
  for (int i = threadIdx.x; i < a.dim; i += kDropThreads) {
    int b = a.nb - 1;
    while (b > 0 && i < a.off[b]) --b;
    chan[i] = (uint16_t)(a.coff[b] + (i - a.off[b]) / a.d[b]);
  }
  const DropKey key = drop_key(a.drop);
  const int chunks = a.dim / V, gl = threadIdx.x & (a.G - 1), group = threadIdx.x / a.G, groups = kDropThreads / a.G;
  for (int64_t t = blockIdx.x; t * a.tile < a.N; t += gridDim.x) {
    const int64_t row0 = t * a.tile;
    const int rows = (int)min((int64_t)a.tile, a.N - row0);
    const uint64_t first = (uint64_t)row0 * a.C;
    const int shift = (int)(first & 3);
    const int blocks = (rows * a.C + shift + 3) / 4;
    __syncthreads();
    for (int i = threadIdx.x; i < blocks; i += kDropThreads) words[i] = keep_bytes(key, a.drop.threshold, (first >> 2) + i);
    __syncthreads();
    for (int r = group; r < rows; r += groups) {
      const unsigned char* keep = reinterpret_cast<const unsigned char*>(words) + shift + r * a.C;
      const float* x = a.x + (row0 + r) * a.dim;
      float* y = a.y + (row0 + r) * a.dim;
      for (int c0 = gl; c0 < chunks; c0 += 4 * a.G) {
        Chunk<V> v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = read_chunk<V>(x + (c0 + i * a.G) * V, c0 + i * a.G < chunks);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = c0 + i * a.G;
          if (c >= chunks) break;
          if constexpr (V == 4) {
            const ushort4 u = *reinterpret_cast<const ushort4*>(chan + 4 * c);
            v[i].x[0] = keep[u.x] ? v[i].x[0] * a.drop.inv_keep : 0.0f;
            v[i].x[1] = keep[u.y] ? v[i].x[1] * a.drop.inv_keep : 0.0f;
            v[i].x[2] = keep[u.z] ? v[i].x[2] * a.drop.inv_keep : 0.0f;
            v[i].x[3] = keep[u.w] ? v[i].x[3] * a.drop.inv_keep : 0.0f;
          } else {
            v[i].x[0] = keep[chan[c]] ? v[i].x[0] * a.drop.inv_keep : 0.0f;
          }
          write_chunk<V>(y + c * V, v[i]);
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

// How a row is spread: lanes G, chunks a lane S (0: neither form takes it), one CTA a row.
struct RowForm {
  int G, S;
  bool cta;
};

RowForm row_form(int dim, int V) {
  const int chunks = dim / V;
  if (chunks > 9 * 32) {
    const int S = (chunks + kRowThreads - 1) / kRowThreads;
    return RowForm{kRowThreads, S <= 2 ? 2 : S <= 4 ? 4 : S <= 8 ? 8 : 0, true};
  }
  RowForm f{32, (chunks + 31) / 32, false};
  // at most four chunks a lane where a row is narrow enough, with as few idle lanes as possible
  for (int G = 16; G >= 1; G /= 2) {
    const int S = (chunks + G - 1) / G;
    if (S <= 4 && G * S < f.G * f.S) f = RowForm{G, S, false};
  }
  if (f.S > 4) f.S = f.S <= 6 ? 6 : 9;
  return f;
}

template <bool BWD, int V, int S, int R, bool CTA>
cudaError_t launch_rows(const NormArgs& a, unsigned grid, cudaStream_t s) {
  const size_t smem = sizeof(float) * 2 * (size_t)a.dim;
  auto kernel = BWD ? k_norm_bwd<V, S, R, CTA> : k_norm_fwd<V, S, R, CTA>;
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, kRowThreads, smem, s>>>(a);
  return cudaGetLastError();
}

// Rows in flight a lane group: enough that a lane has at least four chunks on their way.
constexpr int rows_at_once(int S) { return S == 1 ? 4 : S == 2 ? 2 : 1; }

template <bool BWD, int V>
cudaError_t launch_form(const NormArgs& a, const RowForm& f, unsigned grid, cudaStream_t s) {
  if (f.cta) {
    switch (f.S) {
      case 2: return launch_rows<BWD, V, 2, 1, true>(a, grid, s);
      case 4: return launch_rows<BWD, V, 4, 1, true>(a, grid, s);
      default: return launch_rows<BWD, V, 8, 1, true>(a, grid, s);
    }
  }
  switch (f.S) {
    case 1: return launch_rows<BWD, V, 1, rows_at_once(1), false>(a, grid, s);
    case 2: return launch_rows<BWD, V, 2, rows_at_once(2), false>(a, grid, s);
    case 3: return launch_rows<BWD, V, 3, rows_at_once(3), false>(a, grid, s);
    case 4: return launch_rows<BWD, V, 4, rows_at_once(4), false>(a, grid, s);
    case 6: return launch_rows<BWD, V, 6, rows_at_once(6), false>(a, grid, s);
    default: return launch_rows<BWD, V, 9, rows_at_once(9), false>(a, grid, s);
  }
}

// CTAs of the backward pass (each leaves a partial of the weight gradients): two a SM, and fewer where
// a lane group would not have two rows.
int norm_ctas(int64_t N, int dim) {
  const RowForm f = row_form(dim, 1);
  const int64_t per = f.cta || f.S == 0 ? 1 : kRowThreads / f.G;
  return (int)std::max<int64_t>(1, std::min<int64_t>((N + 2 * per - 1) / (2 * per), kNormMaxCtas));
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace tp

using namespace tp;

struct tp_norm_s {
  NormArgs proto;
  bool vec4;                 // every block's length is a multiple of four floats
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
  if (!((float)eps > 0.0f && (float)eps <= 3.0e38f)) return set_failure(TP_ERR_INVALID_ARG, "eps must be positive and finite");
  a.eps = (float)eps;
  int off = 0;
  bool vec4 = true;
  for (const IrrepTerm& b : t) {
    const int i = a.nb++;
    vec4 = vec4 && b.mul * (2 * b.l + 1) % 4 == 0;
    a.off[i] = off;
    a.mul[i] = b.mul;
    a.d[i] = 2 * b.l + 1;
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
  h->vec4 = vec4;
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
  *bytes = op == TP_OP_FWD ? 0 : sizeof(float) * 2 * (size_t)norm->proto.dim * (size_t)norm_ctas(N, norm->proto.dim);
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
  const int V = norm->vec4 && al16(x) && al16(y) ? 4 : 1;
  const RowForm f = row_form(a.dim, V);
  a.G = f.G;
  count_launches(1);
  if (f.S == 0) {
    k_norm_any<false><<<(unsigned)std::min<int64_t>(N, 148 * 16), kNormThreads, 0, s>>>(a);
    return cuda_status(cudaGetLastError(), "tp_norm_fwd");
  }
  const int64_t per = (f.cta ? 1 : kRowThreads / f.G) * rows_at_once(f.cta ? 3 : f.S);
  const unsigned grid = (unsigned)std::min<int64_t>((N + per - 1) / per, 148 * 8);
  return cuda_status(V == 4 ? launch_form<false, 4>(a, f, grid, s) : launch_form<false, 1>(a, f, grid, s), "tp_norm_fwd");
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
  a.ctas = norm_ctas(N, a.dim);
  const size_t need = sums ? sizeof(float) * 2 * (size_t)a.dim * (size_t)a.ctas : 0;
  if (sums && (!ws || ws_bytes < need)) return set_failure(TP_ERR_WORKSPACE, "workspace too small");
  a.part = sums ? static_cast<float*>(ws) : nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int V = norm->vec4 && al16(x) && al16(gy) && al16(gx) ? 4 : 1;
  const RowForm f = row_form(a.dim, V);
  a.G = f.G;
  cudaError_t e = cudaSuccess;
  count_launches(1);
  if (f.S == 0) {
    const int smem = sums ? (int)(sizeof(float) * 2 * a.dim) : 0;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(k_norm_any<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_status(e, "tp_norm_bwd");
    k_norm_any<true><<<a.ctas, kNormThreads, smem, s>>>(a);
    e = cudaGetLastError();
  } else {
    e = V == 4 ? launch_form<true, 4>(a, f, (unsigned)a.ctas, s) : launch_form<true, 1>(a, f, (unsigned)a.ctas, s);
  }
  if (e == cudaSuccess && sums) {
    unsigned tiles = 0;
    for (int b = 0; b < a.nb; ++b) tiles += (unsigned)((a.mul[b] + 31) / 32) * (a.boff[b] >= 0 ? 2 : 1);
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
  // tiles of up to 4,096 choices, and no larger than leaves four a SM
  a.tile = (int)std::max<int64_t>(1, std::min<int64_t>({64, kDropMaxWords / a.C, N / (148 * 4)}));
  const bool vec4 = a.dim % 4 == 0 && al16(x) && al16(y);
  const int chunks = vec4 ? a.dim / 4 : a.dim;
  a.G = 1;
  while (a.G < 32 && a.G < chunks) a.G *= 2;
  const size_t smem = ((2 * (size_t)a.dim + 15) & ~(size_t)15) + 4 * (((size_t)a.tile * a.C + 3) / 4 + 1);
  const int64_t tiles = (N + a.tile - 1) / a.tile;
  const unsigned grid = (unsigned)std::min<int64_t>(tiles, 148 * 8);
  if (vec4) k_dropout<4><<<grid, kDropThreads, smem, s>>>(a);
  else k_dropout<1><<<grid, kDropThreads, smem, s>>>(a);
  count_launches(1);
  return cuda_status(cudaGetLastError(), "tp_dropout");
}

tp_status_t tp_dropout_bwd(tp_dropout_t drop, int64_t N, const float* gy, double p, const int64_t* rng, int64_t site,
                           float* gx, tp_stream_t stream) {
  return tp_dropout_fwd(drop, N, gy, p, rng, site, gx, stream);
}

}  // extern "C"
