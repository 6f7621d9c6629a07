// Layer normalisation and channel dropout of irreps rows (include/tp_block.h).
//
// Norm, first form: one CTA per row in turn, every thread owning the floats tid, tid + T, ... of
// each block, so that a thread's sums over rows stay its own.  Three reads of a row (mean,
// square, result) come from L1 after the first.
#include <algorithm>
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
constexpr int kNormMaxCtas = 148 * 4;

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
};

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

// gweight[u] = sum over CTAs (in order) and m; gbias likewise.  One warp per output: lanes take
// every 32nd CTA, then join; 64-bit sums, the partials being up to a few hundred terms of both signs.
__global__ void __launch_bounds__(128) k_norm_sums(const __grid_constant__ NormArgs a) {
  const int o = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (o >= a.n_weights + a.n_bias) return;
  const bool bias = o >= a.n_weights;
  float* out = bias ? a.gbias : a.gweight;
  if (!out) return;
  int b = 0;
  const int u = bias ? o - a.n_weights : o;
  if (bias) {
    for (int i = 0; i < a.nb; ++i)
      if (a.boff[i] >= 0 && u >= a.boff[i]) b = i;
  } else {
    while (b + 1 < a.nb && u >= a.woff[b + 1]) ++b;
  }
  const int d = bias ? 1 : a.d[b];
  const int at = (bias ? a.dim : 0) + a.off[b] + (u - (bias ? a.boff[b] : a.woff[b])) * d;
  double t = 0.0;
  for (int c = lane; c < a.ctas; c += 32)
    for (int m = 0; m < d; ++m) t += (double)a.part[(int64_t)c * 2 * a.dim + at + m];
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) t += __shfl_xor_sync(0xffffffffu, t, s);
  if (lane == 0) out[u] = (float)t;
}

// Dropout: a CTA takes a tile of consecutive rows, draws the choices of their channels into
// shared memory (one generator block for four channels) and then passes over the tile's floats.
constexpr int kDropThreads = 256;
constexpr int kDropMaxWords = 4096;    // channels of a tile

struct DropoutArgs {
  int64_t N;
  int dim, C, nb, tile;                // rows per tile
  int off[kNormMaxBlocks], d[kNormMaxBlocks], coff[kNormMaxBlocks];
  const float* x;
  float* y;
  DropArgs drop;
};

__global__ void __launch_bounds__(kDropThreads) k_dropout(const __grid_constant__ DropoutArgs a) {
  extern __shared__ __align__(16) unsigned char sm[];
  uint32_t* words = reinterpret_cast<uint32_t*>(sm);                       // keep bytes, four a word
  uint16_t* chan = reinterpret_cast<uint16_t*>(sm + 4 * (((size_t)a.tile * a.C + 3) / 4 + 1));
  for (int i = threadIdx.x; i < a.dim; i += kDropThreads) {
    int b = a.nb - 1;
    while (b > 0 && i < a.off[b]) --b;
    chan[i] = (uint16_t)(a.coff[b] + (i - a.off[b]) / a.d[b]);
  }
  const DropKey key = drop_key(a.drop);
  for (int64_t t = blockIdx.x; t * a.tile < a.N; t += gridDim.x) {
    const int64_t row0 = t * a.tile;
    const int rows = (int)min((int64_t)a.tile, a.N - row0);
    const uint64_t first = (uint64_t)row0 * a.C;
    const int shift = (int)(first & 3);
    const int blocks = (rows * a.C + shift + 3) / 4;
    __syncthreads();
    for (int i = threadIdx.x; i < blocks; i += kDropThreads) words[i] = keep_bytes(key, a.drop.threshold, (first >> 2) + i);
    __syncthreads();
    const unsigned char* keep = sm + shift;
    const float* x = a.x + row0 * a.dim;
    float* y = a.y + row0 * a.dim;
    const int total = rows * a.dim;
    for (int i = threadIdx.x; i < total; i += kDropThreads) {
      const int r = i / a.dim;
      y[i] = keep[r * a.C + chan[i - r * a.dim]] ? x[i] * a.drop.inv_keep : 0.0f;
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

int norm_ctas(int64_t N) { return (int)std::max<int64_t>(1, std::min<int64_t>(N, kNormMaxCtas)); }

}  // namespace
}  // namespace tp

using namespace tp;

struct tp_norm_s {
  NormArgs proto;
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
  for (const IrrepTerm& b : t) {
    const int i = a.nb++;
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
  *bytes = op == TP_OP_FWD ? 0 : sizeof(float) * 2 * (size_t)norm->proto.dim * (size_t)norm_ctas(N);
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
  k_norm_any<false><<<(unsigned)std::min<int64_t>(N, 148 * 16), kNormThreads, 0, s>>>(a);
  count_launches(1);
  return cuda_status(cudaGetLastError(), "tp_norm_fwd");
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
  a.ctas = norm_ctas(N);
  const size_t need = sums ? sizeof(float) * 2 * (size_t)a.dim * (size_t)a.ctas : 0;
  if (sums && (!ws || ws_bytes < need)) return set_failure(TP_ERR_WORKSPACE, "workspace too small");
  a.part = sums ? static_cast<float*>(ws) : nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int smem = sums ? (int)(sizeof(float) * 2 * a.dim) : 0;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024) e = cudaFuncSetAttribute(k_norm_any<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_status(e, "tp_norm_bwd");
  k_norm_any<true><<<a.ctas, kNormThreads, smem, s>>>(a);
  count_launches(1);
  e = cudaGetLastError();
  if (e == cudaSuccess && sums) {
    k_norm_sums<<<(a.n_weights + a.n_bias + 3) / 4, 128, 0, s>>>(a);
    count_launches(1);
    e = cudaGetLastError();
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
  a.tile = std::max(1, std::min(64, kDropMaxWords / a.C));
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
  const size_t smem = 4 * (((size_t)a.tile * a.C + 3) / 4 + 1) + 2 * (size_t)a.dim;
  const int64_t tiles = (N + a.tile - 1) / a.tile;
  k_dropout<<<(unsigned)std::min<int64_t>(tiles, 148 * 8), kDropThreads, smem, s>>>(a);
  count_launches(1);
  return cuda_status(cudaGetLastError(), "tp_dropout");
}

tp_status_t tp_dropout_bwd(tp_dropout_t drop, int64_t N, const float* gy, double p, const int64_t* rng, int64_t site,
                           float* gx, tp_stream_t stream) {
  return tp_dropout_fwd(drop, N, gy, p, rng, site, gx, stream);
}

}  // extern "C"
