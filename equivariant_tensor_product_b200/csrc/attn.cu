// Equivariant neighbour attention (include/tp_attn.h): softmax over each receiver's edges, with a
// bias per distance bucket and dropout of the probabilities, and its backward pass.
//
// Mapping.  A head's floats (its part of every irreps block) are cut into chunks of V = 4 (or 1)
// floats and dealt to a group of G lanes, S chunks a lane, so that a lane's chunks of q, of the
// accumulators and of the gathered rows stay in registers and a dot product ends in log2 G
// shuffles.  A warp holds 32 / G heads of one receiver; heads beyond 1,024 floats take a whole
// CTA (WIDE), whose dot products are joined through shared memory.
//
// Forward and the receiver pass of the backward walk the edges of a receiver: the senders and
// buckets of 32 edges are read by the 32 lanes, edges that take no part are struck out by a
// ballot, and the rest goes U edges at a time, with all 2 U row gathers issued before the first
// use.  The softmax runs in one pass with the running maximum and sum.
//
// Long rows.  A receiver (sender) of more than `hub` edges would keep one warp busy long after the
// others are done.  Its edges are taken window by window instead: the edge axis is cut into
// windows of win = hub / 2 edges, one CTA each, behind the CTAs of the rows.  A window meets at
// most two such rows (the row of its first edge and the row of its last one), finds them by a
// 33-way search in the row pointers and leaves a partial row for each; k_attn_join adds a row's
// partials up in window order.  Graphs of at most `hub` edges have neither windows nor the join.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>
#include <vector>

#include "../../include/tp_attn.h"
#include "philox.cuh"
#include "tp_common.h"
#include "tp_host.h"

namespace tp {
namespace {

constexpr int kAttnMaxBlocks = 16;
constexpr int kAttnThreads = 128;
constexpr int kAttnWarps = kAttnThreads / 32;
constexpr int kAttnWideThreads = 512;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

// Where a head's floats lie in a row: len[b] floats from off[b] + h len[b] on, block after block.
struct HeadMap {
  int nb, hd;
  int off[kAttnMaxBlocks], len[kAttnMaxBlocks];
};

struct AttnArgs {
  int N, E, H, K;
  int hw, groups;            // heads per warp (a power of two), head groups of a row
  int W;                     // warps that split a row's edges
  int row_ctas;              // CTAs of the rows; the windows' CTAs come after them
  int hub, win, n_win;       // rows of more than hub edges go by windows (n_win = 0: no such rows)
  float* part;               // workspace [n_win][2][part_len]: partial rows of the windows
  int part_len;
  int dq, dv;
  const int32_t* rowptr;
  const int32_t* src;
  const int32_t* colptr;
  const int32_t* perm;
  const int32_t* bucket;
  const float* q;
  const float* k;
  const float* v;
  int64_t ldq, ldk, ldv;
  const float* table;
  float scale;
  DropArgs drop;
  const float* y_in;
  const float* lse_in;
  const float* gy;
  float* y;
  float* lse;
  float* gq;
  float* gk;
  float* gv;
  int64_t ldgq, ldgk, ldgv;
  float* gtable;
  float2* rec;               // workspace [E][H]: (ds, r p) of the backward pass
  int32_t* dst;              // workspace [E]: receiver, -1 for an edge that takes no part
  float* hist;               // workspace [hist_ctas][K * H]
  int hist_ctas, hist_copies, hist_lanes;
  HeadMap mq, mv;
};

constexpr int kMinWindow = 128;

__device__ __forceinline__ int slot_offset(const HeadMap& m, int h, int pos) {
  for (int b = 0; b < m.nb; ++b) {
    if (pos < m.len[b]) return m.off[b] + h * m.len[b] + pos;
    pos -= m.len[b];
  }
  return -1;
}

template <int V>
struct Vec {
  float x[V];
};

template <int V>
__device__ __forceinline__ Vec<V> load_vec(const float* p, bool on) {
  Vec<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.x[i] = 0.0f;
  if (on) {
    if constexpr (V == 4) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(p));
      r.x[0] = t.x, r.x[1] = t.y, r.x[2] = t.z, r.x[3] = t.w;
    } else {
      r.x[0] = __ldg(p);
    }
  }
  return r;
}

template <int V>
__device__ __forceinline__ void store_vec(float* p, const Vec<V>& r) {
  if constexpr (V == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(r.x[0], r.x[1], r.x[2], r.x[3]);
  } else {
    *p = r.x[0];
  }
}

__device__ __forceinline__ float exp_of(float x) { return exp2f(x * kLog2e); }

__device__ __forceinline__ int clamp_edge(int e, int E) { return min(max(e, 0), E); }

// The row r of `ptr` with ptr[r] <= e < ptr[r + 1], or -1: 32 probes a step, the same answer in every lane.
__device__ __forceinline__ int find_row(const int32_t* __restrict__ ptr, int N, int e) {
  if (e < __ldg(ptr) || e >= __ldg(ptr + N)) return -1;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int step = (hi - lo + 32) / 33;
    const int64_t pos = lo + (int64_t)(lane + 1) * step;
    const int below = __popc(__ballot_sync(kFull, pos < hi && __ldg(ptr + min(pos, (int64_t)hi)) <= e));
    lo += below * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// A stretch of one row's edges that a CTA's warps work on: a whole row, or a window's share of a long one.
struct Task {
  int row, head0, split, W, lo, hi;
  float* part;               // where a window leaves its partial row
  bool write;                // false: a long row, which the windows deal with
};

// Number of tasks of this CTA.  Rows: one.  Windows: the heads of up to two rows, found here.
struct Tasks {
  int n, first, row0, row1;

  __device__ __forceinline__ Tasks(const AttnArgs& a, const int32_t* __restrict__ ptr, bool wide) {
    __shared__ int found[2];
    n = 1;
    if ((int)blockIdx.x < a.row_ctas) return;
    first = ((int)blockIdx.x - a.row_ctas) * a.win;
    if (threadIdx.x < 64) {
      const int slot = threadIdx.x >> 5;
      int r = find_row(ptr, a.N, slot ? min(first + a.win, a.E) - 1 : first);
      if (r >= 0) {
        const int start = __ldg(ptr + r);
        if (__ldg(ptr + r + 1) - start <= a.hub || (slot && start <= first)) r = -1;
      }
      if ((threadIdx.x & 31) == 0) found[slot] = r;
    }
    __syncthreads();
    row0 = found[0];
    row1 = found[1];
    n = 2 * (wide ? a.H : a.groups);
  }

  __device__ __forceinline__ Task get(const AttnArgs& a, const int32_t* __restrict__ ptr, int i, bool wide) const {
    Task t;
    const int warp = threadIdx.x >> 5;
    t.part = nullptr;
    t.write = false;
    t.row = a.N;
    t.lo = t.hi = t.head0 = t.split = 0;
    t.W = 1;
    if ((int)blockIdx.x < a.row_ctas) {
      if (wide) {
        t.row = blockIdx.x / a.H;
        t.head0 = blockIdx.x - t.row * a.H;
      } else {
        const int unit = blockIdx.x * (kAttnWarps / a.W) + warp / a.W;
        t.W = a.W;
        t.split = warp % a.W;
        t.row = unit / a.groups;
        t.head0 = (unit - t.row * a.groups) * a.hw;
      }
      if (t.row >= a.N) return t;
      t.lo = clamp_edge(__ldg(ptr + t.row), a.E);
      t.hi = clamp_edge(__ldg(ptr + t.row + 1), a.E);
      t.write = a.n_win == 0 || t.hi - t.lo <= a.hub;
      if (!t.write) t.hi = t.lo;
    } else {
      const int per = wide ? a.H : a.groups, slot = i / per;
      const int r = slot ? row1 : row0;
      if (r < 0) return t;
      t.row = r;
      t.head0 = (i - slot * per) * (wide ? 1 : a.hw);
      t.write = true;
      t.part = a.part + ((int64_t)((int)blockIdx.x - a.row_ctas) * 2 + slot) * a.part_len;
      t.lo = max(__ldg(ptr + t.row), first);
      t.hi = min(min(__ldg(ptr + t.row + 1), first + a.win), a.E);
      if (!wide) {
        t.W = kAttnWarps;
        t.split = warp;
      }
    }
    if (t.W > 1 && t.hi > t.lo) {
      const int per = (t.hi - t.lo + t.W - 1) / t.W;
      t.lo += min(t.split * per, t.hi - t.lo);
      t.hi = min(t.hi, t.lo + per);
    }
    return t;
  }
};

// Which head and chunks of the task's row a thread holds.
template <int V, int S, bool WIDE>
struct Lane {
  int h, G, gl, sub;
  bool live;                 // the lane holds a head of a row
  int oq[S], ov[S];

  __device__ __forceinline__ Lane(const AttnArgs& a, const Task& t) {
    const int lane = threadIdx.x & 31;
    if constexpr (WIDE) {
      h = t.head0;
      sub = 0;
      G = blockDim.x;
      gl = threadIdx.x;
    } else {
      G = 32 / a.hw;
      sub = lane / G;
      gl = lane & (G - 1);
      h = t.head0 + sub;
    }
    live = t.write && t.row < a.N && h < a.H;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int pos = (s * G + gl) * V;
      oq[s] = live ? slot_offset(a.mq, h, pos) : -1;
      ov[s] = live ? slot_offset(a.mv, h, pos) : -1;
    }
  }

  // Sums of U values over the group, in every lane of it.  WIDE: `buf` holds [2][warps][U], used in turn.
  template <int U>
  __device__ __forceinline__ void sum(float (&v)[U], float* buf, int& turn) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (WIDE || G > o) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] += __shfl_xor_sync(kFull, v[u], o);
      }
    if constexpr (WIDE) {
      float* b = buf + turn * (kAttnWideThreads / 32) * U;
      turn ^= 1;
      if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) b[(threadIdx.x >> 5) * U + u] = v[u];
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = 0.0f;
      for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] += b[w * U + u];
      }
    }
  }
};

// One lane's edge of a batch of 32: sender (-1: takes no part), bucket, and a bit per head of the warp
// that is set where dropout keeps the probability.
struct EdgeLane {
  int j, b;
  uint32_t keep;
};

__device__ __forceinline__ EdgeLane read_edge(const AttnArgs& a, const DropKey& key, int e, bool on, int head0, int heads) {
  EdgeLane r{-1, 0, ~0u};
  if (on) {
    r.j = __ldg(a.src + e);
    if ((unsigned)r.j >= (unsigned)a.N) r.j = -1;
    if (a.bucket) {
      r.b = __ldg(a.bucket + e);
      if ((unsigned)r.b >= (unsigned)a.K) r.j = -1;
    }
    if (a.drop.rng && r.j >= 0) {
      r.keep = 0;
      const uint64_t first = (uint64_t)e * a.H + head0;
      for (uint64_t blk = first >> 2; blk * 4 < first + heads; ++blk) {
        const uint32_t k = keep_bytes(key, a.drop.threshold, blk);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int w = (int)(int64_t)(blk * 4 + i - first);
          if (w >= 0 && w < heads) r.keep |= ((k >> (8 * i)) & 1u) << w;
        }
      }
    }
  }
  return r;
}

template <int V, int S, int U, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kAttnWideThreads : kAttnThreads) k_attn_fwd(const __grid_constant__ AttnArgs a) {
  __shared__ float join[WIDE ? 2 * (kAttnWideThreads / 32) * U : kAttnWarps * (V * S + 2) * 32];
  const int lane = threadIdx.x & 31;
  int turn = 0;
  DropKey key{};
  if (a.drop.rng) key = drop_key(a.drop);
  const Tasks tasks(a, a.rowptr, WIDE);
  for (int task = 0; task < tasks.n; ++task) {
  const Task t = tasks.get(a, a.rowptr, task, WIDE);
  const Lane<V, S, WIDE> L(a, t);
  Vec<V> q[S], acc[S];
  float m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    q[s] = load_vec<V>(a.q + (int64_t)t.row * a.ldq + L.oq[s], L.oq[s] >= 0);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[s].x[i] = 0.0f;
  }
  for (int base = t.lo; base < t.hi; base += 32) {
    const EdgeLane mine = read_edge(a, key, base + lane, base + lane < t.hi, t.head0, WIDE ? 1 : a.hw);
    uint32_t left = __ballot_sync(kFull, mine.j >= 0);
    while (left) {
      Vec<V> kk[U][S], vv[U][S];
      float bias[U], dot[U];
      bool kept[U], on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = left ? __ffs(left) - 1 : 0;
        on[u] = left != 0;
        left &= left - 1;
        const int64_t j = __shfl_sync(kFull, mine.j, at);
        const int b = __shfl_sync(kFull, mine.b, at);
        kept[u] = (__shfl_sync(kFull, mine.keep, at) >> L.sub) & 1u;
#pragma unroll
        for (int s = 0; s < S; ++s) kk[u][s] = load_vec<V>(a.k + j * a.ldk + L.oq[s], on[u] && L.oq[s] >= 0);
#pragma unroll
        for (int s = 0; s < S; ++s) vv[u][s] = load_vec<V>(a.v + j * a.ldv + L.ov[s], on[u] && L.ov[s] >= 0);
        bias[u] = 0.0f;
        if (a.table && on[u] && L.live) bias[u] = __ldg(a.table + (int64_t)b * a.H + L.h);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        dot[u] = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) dot[u] = fmaf(q[s].x[i], kk[u][s].x[i], dot[u]);
      }
      L.sum(dot, join, turn);
      float top = m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool out = !on[u] || bias[u] == -INFINITY;
        dot[u] = out ? -INFINITY : fmaf(dot[u], a.scale, bias[u]);
        if (out) {                       // a masked row may hold anything: 0 times it has to be 0
#pragma unroll
          for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) vv[u][s].x[i] = 0.0f;
        }
        top = fmaxf(top, dot[u]);
      }
      const float ref = top == -INFINITY ? 0.0f : top;
      const float shrink = exp_of(m - ref);
      m = top;
      l *= shrink;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[s].x[i] *= shrink;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float p = exp_of(dot[u] - ref);
        l += p;
        const float pr = kept[u] ? p : 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) acc[s].x[i] = fmaf(pr, vv[u][s].x[i], acc[s].x[i]);
      }
    }
  }
  if constexpr (!WIDE) {
    if (t.W > 1) {                       // join the warps of a row in order
      const int warp = threadIdx.x >> 5;
      float* mine = join + warp * (V * S + 2) * 32;
      if (t.split > 0) {
        mine[lane] = m;
        mine[32 + lane] = l;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) mine[(2 + s * V + i) * 32 + lane] = acc[s].x[i];
      }
      __syncthreads();
      for (int w = 1; t.split == 0 && w < t.W; ++w) {
        const float* other = join + (warp + w) * (V * S + 2) * 32;
        const float m2 = other[lane], top = fmaxf(m, m2), ref = top == -INFINITY ? 0.0f : top;
        const float f1 = exp_of(m - ref), f2 = exp_of(m2 - ref);
        l = l * f1 + other[32 + lane] * f2;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) acc[s].x[i] = acc[s].x[i] * f1 + other[(2 + s * V + i) * 32 + lane] * f2;
        m = top;
      }
    }
  }
  if (L.live && t.split == 0) {
    if (t.part) {
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (L.ov[s] >= 0) store_vec<V>(t.part + L.ov[s], acc[s]);
      if (L.gl == 0) {
        t.part[a.part_len - 2 * a.H + L.h] = m;
        t.part[a.part_len - a.H + L.h] = l;
      }
    } else {
      const bool none = m == -INFINITY && l == 0.0f;
      const float f = none ? 0.0f : a.drop.inv_keep / l;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (L.ov[s] < 0) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[s].x[i] *= f;
        store_vec<V>(a.y + (int64_t)t.row * a.dv + L.ov[s], acc[s]);
      }
      if (a.lse && L.gl == 0) a.lse[(int64_t)t.row * a.H + L.h] = none ? -INFINITY : m + logf(l);
    }
  }
  if (task + 1 < tasks.n) __syncthreads();   // the join buffer is free again
  }
}

// Backward, receiver order: gq, and for the sender pass and gtable (ds, r p) of every edge and head
// and the receiver of every edge.
template <int V, int S, int U, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kAttnWideThreads : kAttnThreads) k_attn_bwd_recv(const __grid_constant__ AttnArgs a) {
  __shared__ float join[WIDE ? 2 * (kAttnWideThreads / 32) * 2 * U : kAttnWarps * V * S * 32];
  const int lane = threadIdx.x & 31;
  int turn = 0;
  DropKey key{};
  if (a.drop.rng) key = drop_key(a.drop);
  const Tasks tasks(a, a.rowptr, WIDE);
  for (int task = 0; task < tasks.n; ++task) {
  const Task t = tasks.get(a, a.rowptr, task, WIDE);
  const Lane<V, S, WIDE> L(a, t);
  Vec<V> q[S], gy[S], acc[S];
  float delta[2 * U];
#pragma unroll
  for (int u = 0; u < 2 * U; ++u) delta[u] = 0.0f;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    q[s] = load_vec<V>(a.q + (int64_t)t.row * a.ldq + L.oq[s], L.oq[s] >= 0);
    gy[s] = load_vec<V>(a.gy + (int64_t)t.row * a.dv + L.ov[s], L.ov[s] >= 0);
    const Vec<V> y = load_vec<V>(a.y_in + (int64_t)t.row * a.dv + L.ov[s], L.ov[s] >= 0);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      acc[s].x[i] = 0.0f;
      delta[0] = fmaf(gy[s].x[i], y.x[i], delta[0]);
    }
  }
  L.sum(delta, join, turn);
  const float del = delta[0];
  const float lse = L.live ? __ldg(a.lse_in + (int64_t)t.row * a.H + L.h) : 0.0f;
  for (int base = t.lo; base < t.hi; base += 32) {
    const EdgeLane mine = read_edge(a, key, base + lane, base + lane < t.hi, t.head0, WIDE ? 1 : a.hw);
    if (a.rec && base + lane < t.hi && t.head0 == 0 && (!WIDE || threadIdx.x < 32))
      a.dst[base + lane] = mine.j >= 0 ? t.row : -1;
    if (a.rec && base + lane < t.hi && mine.j < 0 && (!WIDE || threadIdx.x < 32))
      for (int h = t.head0; h < min(a.H, t.head0 + (WIDE ? 1 : a.hw)); ++h)
        a.rec[(int64_t)(base + lane) * a.H + h] = make_float2(0.0f, 0.0f);
    uint32_t left = __ballot_sync(kFull, mine.j >= 0);
    while (left) {
      Vec<V> kk[U][S], vv[U][S];
      float bias[U], dot[2 * U];
      bool kept[U], on[U];
      int at[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        at[u] = left ? __ffs(left) - 1 : 0;
        on[u] = left != 0;
        left &= left - 1;
        const int64_t j = __shfl_sync(kFull, mine.j, at[u]);
        const int b = __shfl_sync(kFull, mine.b, at[u]);
        kept[u] = (__shfl_sync(kFull, mine.keep, at[u]) >> L.sub) & 1u;
#pragma unroll
        for (int s = 0; s < S; ++s) kk[u][s] = load_vec<V>(a.k + j * a.ldk + L.oq[s], on[u] && L.oq[s] >= 0);
#pragma unroll
        for (int s = 0; s < S; ++s) vv[u][s] = load_vec<V>(a.v + j * a.ldv + L.ov[s], on[u] && L.ov[s] >= 0);
        bias[u] = 0.0f;
        if (a.table && on[u] && L.live) bias[u] = __ldg(a.table + (int64_t)b * a.H + L.h);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        dot[u] = dot[U + u] = 0.0f;
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            dot[u] = fmaf(q[s].x[i], kk[u][s].x[i], dot[u]);
            dot[U + u] = fmaf(gy[s].x[i], vv[u][s].x[i], dot[U + u]);
          }
      }
      L.sum(dot, join, turn);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool out = !on[u] || bias[u] == -INFINITY || lse == -INFINITY;
        const float p = out ? 0.0f : exp_of(fmaf(dot[u], a.scale, bias[u]) - lse);
        const float r = kept[u] ? a.drop.inv_keep : 0.0f;
        const float ds = out ? 0.0f : p * (r * dot[U + u] - del);
        if (out) {
#pragma unroll
          for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) kk[u][s].x[i] = 0.0f;
        }
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) acc[s].x[i] = fmaf(ds, kk[u][s].x[i], acc[s].x[i]);
        if (a.rec && on[u] && L.live && L.gl == 0)
          a.rec[(int64_t)(base + at[u]) * a.H + L.h] = make_float2(ds, p * r);
      }
    }
  }
  if constexpr (!WIDE) {
    if (t.W > 1) {
      const int warp = threadIdx.x >> 5;
      if (t.split > 0) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) join[(warp * S * V + s * V + i) * 32 + lane] = acc[s].x[i];
      }
      __syncthreads();
      for (int w = 1; t.split == 0 && w < t.W; ++w)
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) acc[s].x[i] += join[((warp + w) * S * V + s * V + i) * 32 + lane];
    }
  }
  if (L.live && t.split == 0 && a.gq) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (L.oq[s] < 0) continue;
      if (t.part) {
        store_vec<V>(t.part + L.oq[s], acc[s]);
        continue;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) acc[s].x[i] *= a.scale;
      store_vec<V>(a.gq + (int64_t)t.row * a.ldgq + L.oq[s], acc[s]);
    }
  }
  if (task + 1 < tasks.n) __syncthreads();   // the join buffer is free again
  }
}

// Backward, sender order: gk[j] = scale sum ds q[i], gv[j] = sum r p gy[i] over the edges that leave j.
template <int V, int S, int U, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kAttnWideThreads : kAttnThreads) k_attn_bwd_send(const __grid_constant__ AttnArgs a) {
  __shared__ float join[WIDE ? 1 : kAttnWarps * 2 * V * S * 32];
  const int lane = threadIdx.x & 31;
  const int e_lo = max(__ldg(a.rowptr), 0), e_hi = min(__ldg(a.rowptr + a.N), a.E);
  const Tasks tasks(a, a.colptr, WIDE);
  for (int task = 0; task < tasks.n; ++task) {
  const Task t = tasks.get(a, a.colptr, task, WIDE);
  const Lane<V, S, WIDE> L(a, t);
  Vec<V> ak[S], av[S];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int i = 0; i < V; ++i) ak[s].x[i] = av[s].x[i] = 0.0f;
  for (int base = t.lo; base < t.hi; base += 32) {
    int e = -1, i = -1;
    if (base + lane < t.hi) {
      e = __ldg(a.perm + base + lane);
      if (e >= e_lo && e < e_hi) i = a.dst[e];
    }
    uint32_t left = __ballot_sync(kFull, i >= 0);
    while (left) {
      Vec<V> qq[U][S], gg[U][S];
      float2 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = left ? __ffs(left) - 1 : 0;
        const bool on = left != 0;
        left &= left - 1;
        const int64_t r = __shfl_sync(kFull, i, at);
        const int64_t ee = __shfl_sync(kFull, e, at);
        w[u] = make_float2(0.0f, 0.0f);
        if (on && L.live) w[u] = a.rec[ee * a.H + L.h];
#pragma unroll
        for (int s = 0; s < S; ++s) qq[u][s] = load_vec<V>(a.q + r * a.ldq + L.oq[s], on && L.oq[s] >= 0);
#pragma unroll
        for (int s = 0; s < S; ++s) gg[u][s] = load_vec<V>(a.gy + r * a.dv + L.ov[s], on && L.ov[s] >= 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (w[u].x == 0.0f && w[u].y == 0.0f) continue;     // no part of this head: 0 times its rows is 0
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i2 = 0; i2 < V; ++i2) {
            ak[s].x[i2] = fmaf(w[u].x, qq[u][s].x[i2], ak[s].x[i2]);
            av[s].x[i2] = fmaf(w[u].y, gg[u][s].x[i2], av[s].x[i2]);
          }
      }
    }
  }
  if constexpr (!WIDE) {
    if (t.W > 1) {
      const int warp = threadIdx.x >> 5;
      if (t.split > 0) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            join[((warp * 2 + 0) * S * V + s * V + i) * 32 + lane] = ak[s].x[i];
            join[((warp * 2 + 1) * S * V + s * V + i) * 32 + lane] = av[s].x[i];
          }
      }
      __syncthreads();
      for (int o = 1; t.split == 0 && o < t.W; ++o)
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            ak[s].x[i] += join[(((warp + o) * 2 + 0) * S * V + s * V + i) * 32 + lane];
            av[s].x[i] += join[(((warp + o) * 2 + 1) * S * V + s * V + i) * 32 + lane];
          }
    }
  }
  if (L.live && t.split == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (t.part) {
        if (L.oq[s] >= 0) store_vec<V>(t.part + L.oq[s], ak[s]);
        if (L.ov[s] >= 0) store_vec<V>(t.part + a.dq + L.ov[s], av[s]);
        continue;
      }
      if (a.gk && L.oq[s] >= 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) ak[s].x[i] *= a.scale;
        store_vec<V>(a.gk + (int64_t)t.row * a.ldgk + L.oq[s], ak[s]);
      }
      if (a.gv && L.ov[s] >= 0) store_vec<V>(a.gv + (int64_t)t.row * a.ldgv + L.ov[s], av[s]);
    }
  }
  if (task + 1 < tasks.n) __syncthreads();   // the join buffer is free again
  }
}

// Joins the partial rows of the long rows, in window order: CTA w acts when such a row begins in window w.
// Its eight warps take every eighth window, 128 floats of the row at a time, and are then added up in
// order.  Forward: the windows' sums meet at their common maximum.  Bound by the reads of the partials,
// one row for `win` edges' gathers of two.
constexpr int kJoinThreads = 256;

template <int PASS>   // 0: y, lse; 1: gq; 2: gk, gv
__device__ __forceinline__ void join_long_row(const AttnArgs& a, int w) {
  __shared__ float top[32], total[32], sums[kJoinThreads / 32][128];
  const int32_t* ptr = PASS == 2 ? a.colptr : a.rowptr;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kJoinThreads / 32;
  const int first = w * a.win, end = min(first + a.win, a.E);
  const int row = find_row(ptr, a.N, end - 1);
  if (row < 0) return;
  const int start = __ldg(ptr + row), stop = min(__ldg(ptr + row + 1), a.E);
  if (start < first || __ldg(ptr + row + 1) - start <= a.hub) return;
  const int n = (stop - 1) / a.win - w + 1;             // windows w .. w + n - 1; only the first may be slot 1
  auto part = [&](int i) {
    return a.part + ((int64_t)(w + i) * 2 + (i == 0 && start > first ? 1 : 0)) * a.part_len;
  };
  if (PASS == 0) {
    for (int h = warp; h < a.H; h += warps) {
      float m = -INFINITY, l = 0.0f;
      for (int i = lane; i < n; i += 32) m = fmaxf(m, part(i)[a.part_len - 2 * a.H + h]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      const float ref = m == -INFINITY ? 0.0f : m;
      for (int i = lane; i < n; i += 32) {
        const float* p = part(i) + a.part_len - 2 * a.H + h;
        l += p[a.H] * exp_of(p[0] - ref);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
      if (lane == 0) {
        top[h] = ref;
        const bool none = m == -INFINITY && l == 0.0f;
        total[h] = none ? 0.0f : a.drop.inv_keep / l;
        if (a.lse) a.lse[(int64_t)row * a.H + h] = none ? -INFINITY : m + logf(l);
      }
    }
    __syncthreads();
  }
  const int width = PASS == 0 ? a.dv : PASS == 1 ? a.dq : a.dq + a.dv;
  for (int d0 = 0; d0 < width; d0 += 128) {
    float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    int head[4] = {0, 0, 0, 0};
    if (PASS == 0) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int d = min(d0 + c * 32 + lane, width - 1);
        int b = a.mv.nb - 1;
        while (b > 0 && d < a.mv.off[b]) --b;
        head[c] = (d - a.mv.off[b]) / a.mv.len[b];
      }
    }
#pragma unroll 4
    for (int i = warp; i < n; i += warps) {
      const float* p = part(i);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int d = d0 + c * 32 + lane;
        if (d >= width) continue;
        const float f = PASS == 0 ? exp_of(p[a.part_len - 2 * a.H + head[c]] - top[head[c]]) : 1.0f;
        t[c] = fmaf(f, p[d], t[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) sums[warp][c * 32 + lane] = t[c];
    __syncthreads();
    const int d = d0 + threadIdx.x;
    if (threadIdx.x < 128 && d < width) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < kJoinThreads / 32; ++i) v += sums[i][threadIdx.x];
      if (PASS == 0) {
        int b = a.mv.nb - 1;
        while (b > 0 && d < a.mv.off[b]) --b;
        a.y[(int64_t)row * a.dv + d] = v * total[(d - a.mv.off[b]) / a.mv.len[b]];
      } else if (PASS == 1) {
        a.gq[(int64_t)row * a.ldgq + d] = a.scale * v;
      } else if (d < a.dq) {
        if (a.gk) a.gk[(int64_t)row * a.ldgk + d] = a.scale * v;
      } else if (a.gv) {
        a.gv[(int64_t)row * a.ldgv + d - a.dq] = v;
      }
    }
    __syncthreads();
  }
}

template <int PASS>
__global__ void __launch_bounds__(kJoinThreads) k_attn_join(const __grid_constant__ AttnArgs a) {
  join_long_row<PASS>(a, blockIdx.x);
}

// gtable[b, h] = sum of ds over the edges of bucket b.  The edges are cut into contiguous ranges, one
// for each group of lanes; a group's lanes own one head each and add into the group's own copy of the
// table in shared memory, edge after edge, so every sum has a fixed order.
__global__ void __launch_bounds__(kAttnThreads) k_attn_table(const __grid_constant__ AttnArgs a) {
  extern __shared__ float copies[];
  const int KH = a.K * a.H, group = threadIdx.x / a.hist_lanes, h = threadIdx.x % a.hist_lanes;
  for (int i = threadIdx.x; i < KH * a.hist_copies; i += kAttnThreads) copies[i] = 0.0f;
  __syncthreads();
  const int lo = max(0, min(__ldg(a.rowptr), a.E)), hi = max(lo, min(__ldg(a.rowptr + a.N), a.E));
  if (group < a.hist_copies && h < a.H) {
    const int64_t ranges = (int64_t)a.hist_ctas * a.hist_copies, r = (int64_t)blockIdx.x * a.hist_copies + group;
    const int first = lo + (int)((hi - lo) * r / ranges), last = lo + (int)((hi - lo) * (r + 1) / ranges);
    float* mine = copies + group * KH;
    for (int e = first; e < last; ++e) {
      const int b = __ldg(a.bucket + e);
      const float ds = a.rec[(int64_t)e * a.H + h].x;
      if ((unsigned)b < (unsigned)a.K) mine[b * a.H + h] += ds;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < KH; i += kAttnThreads) {
    float t = 0.0f;
    for (int c = 0; c < a.hist_copies; ++c) t += copies[c * KH + i];
    (a.hist_ctas == 1 ? a.gtable : a.hist + (int64_t)blockIdx.x * KH)[i] = t;
  }
}

__global__ void __launch_bounds__(128) k_attn_table_sum(const __grid_constant__ AttnArgs a) {
  const int KH = a.K * a.H, o = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (o >= KH) return;
  double t = 0.0;
  for (int c = lane; c < a.hist_ctas; c += 32) t += (double)a.hist[(int64_t)c * KH + o];
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) t += __shfl_xor_sync(kFull, t, s);
  if (lane == 0) a.gtable[o] = (float)t;
}

// Distance buckets: squares in 64 bits (products of 32-bit floats are exact there), binary search.
constexpr int kMaxBounds = 1023;

__global__ void __launch_bounds__(256) k_buckets(int64_t E, const float* __restrict__ vec, int n, const float* __restrict__ bounds,
                                                 double cut2, int32_t* __restrict__ bucket) {
  __shared__ double b2[kMaxBounds + 1];
  for (int i = threadIdx.x; i < n; i += 256) {
    const double b = (double)bounds[i];
    b2[i] = b < 0.0 ? -1.0 : b * b;
  }
  __syncthreads();
  for (int64_t e = blockIdx.x * (int64_t)256 + threadIdx.x; e < E; e += (int64_t)gridDim.x * 256) {
    const double x = vec[3 * e], y = vec[3 * e + 1], z = vec[3 * e + 2];
    const double d2 = x * x + y * y + z * z;
    int lo = 0, hi = n;                  // the first bound above the distance lies in [lo, hi]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (d2 >= b2[mid]) lo = mid + 1;
      else hi = mid;
    }
    bucket[e] = d2 < cut2 ? lo : -1;
  }
}

// ---------------------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------------------

bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t al256(size_t v) { return (v + 255) & ~size_t(255); }
tp_status_t cuda_status(cudaError_t e, const char* where) {
  return e == cudaSuccess ? TP_OK : set_failure(TP_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

enum Pass { kFwd, kRecv, kSend };

template <int V, int S, int U, bool WIDE>
void launch_one(Pass pass, const AttnArgs& a, unsigned grid, int threads, cudaStream_t s) {
  if (pass == kFwd) k_attn_fwd<V, S, U, WIDE><<<grid, threads, 0, s>>>(a);
  else if (pass == kRecv) k_attn_bwd_recv<V, S, U, WIDE><<<grid, threads, 0, s>>>(a);
  else k_attn_bwd_send<V, S, U, WIDE><<<grid, threads, 0, s>>>(a);
}

// Chunks a lane holds at most; the kernels exist for these counts.
int slots_for(int need, bool wide) {
  for (int s : {1, 2, 3, 4, 6, 8})
    if (need <= s && !(wide && (s == 1 || s == 3 || s == 6))) return s;
  return 0;
}

template <int V>
void launch_slots(Pass pass, AttnArgs& a, cudaStream_t s) {
  const int chunks = (std::max(a.mq.hd, a.mv.hd) + V - 1) / V;
  if (chunks > 256) {
    int threads = 128;
    while (threads < kAttnWideThreads && (chunks + threads - 1) / threads > 4) threads *= 2;
    a.hw = 1;
    a.groups = a.H;
    a.W = 1;
    a.row_ctas = a.N * a.H;
    const unsigned grid = (unsigned)(a.row_ctas + a.n_win);
    switch (slots_for((chunks + threads - 1) / threads, true)) {
      case 2: return launch_one<V, 2, 4, true>(pass, a, grid, threads, s);
      case 4: return launch_one<V, 4, 2, true>(pass, a, grid, threads, s);
      default: return launch_one<V, 8, 1, true>(pass, a, grid, threads, s);
    }
  }
  // as many heads in a warp as leave a lane at most four chunks
  int hw = 1;
  while (hw < a.H && (chunks * 2 * hw + 31) / 32 <= 4) hw *= 2;
  a.hw = hw;
  a.groups = (a.H + hw - 1) / hw;
  const int need = (chunks + 32 / hw - 1) / (32 / hw);
  const int64_t units = (int64_t)a.N * a.groups;
  a.W = 1;
  while (a.W < kAttnWarps && units * a.W < 148 * 24 && a.E / std::max(1, a.N) >= 8 * a.W) a.W *= 2;
  const int per = kAttnWarps / a.W;
  a.row_ctas = (int)((units + per - 1) / per);
  const unsigned grid = (unsigned)(a.row_ctas + a.n_win);
  switch (slots_for(need, false)) {
    case 1: return launch_one<V, 1, 4, false>(pass, a, grid, kAttnThreads, s);
    case 2: return launch_one<V, 2, 4, false>(pass, a, grid, kAttnThreads, s);
    case 3: return launch_one<V, 3, 2, false>(pass, a, grid, kAttnThreads, s);
    case 4: return launch_one<V, 4, 2, false>(pass, a, grid, kAttnThreads, s);
    case 6: return launch_one<V, 6, 1, false>(pass, a, grid, kAttnThreads, s);
    default: return launch_one<V, 8, 1, false>(pass, a, grid, kAttnThreads, s);
  }
}

// Windows of at least 128 edges, and no more of them than 16 a SM: rows of up to twice that stay with
// their own warps.
void window_plan(AttnArgs& a) {
  a.win = std::max(kMinWindow, (a.E / (148 * 16) + 32) / 32 * 32);
  a.hub = 2 * a.win;
  a.n_win = a.E > a.hub ? (a.E + a.win - 1) / a.win : 0;
}

int part_len(const AttnArgs& a, Pass pass) {
  const int n = pass == kFwd ? a.dv + 2 * a.H : pass == kRecv ? a.dq : a.dq + a.dv;
  return (n + 3) & ~3;
}

size_t part_bytes(const AttnArgs& a, Pass pass) { return sizeof(float) * 2 * (size_t)a.n_win * part_len(a, pass); }

cudaError_t launch_pass(Pass pass, AttnArgs& a, bool vec4, float* part, cudaStream_t s) {
  a.part = part;
  a.part_len = part_len(a, pass);
  if (vec4) launch_slots<4>(pass, a, s);
  else launch_slots<1>(pass, a, s);
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.n_win == 0 || (pass == kRecv && !a.gq)) return e;
  if (pass == kFwd) k_attn_join<0><<<a.n_win, kJoinThreads, 0, s>>>(a);
  else if (pass == kRecv) k_attn_join<1><<<a.n_win, kJoinThreads, 0, s>>>(a);
  else k_attn_join<2><<<a.n_win, kJoinThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

void hist_plan(AttnArgs& a) {
  a.hist_lanes = 1;
  while (a.hist_lanes < a.H) a.hist_lanes *= 2;
  const int KH = std::max(1, a.K * a.H);
  a.hist_copies = std::max(1, std::min(kAttnThreads / a.hist_lanes, 24 * 1024 / KH));
  // a CTA zeroes, sums and writes KH floats: give it at least as many edges' values
  const int64_t want = std::max<int64_t>(1, (int64_t)a.E / std::max(1024, KH / a.H * 4));
  a.hist_ctas = (int)std::min<int64_t>(want, 148 * 2);
}

}  // namespace
}  // namespace tp

using namespace tp;

struct tp_attn_s {
  AttnArgs proto;
  bool vec4;                 // every head's floats of every block are a multiple of four
};

namespace {

struct BwdLayout {
  size_t rec, dst, hist, colptr, perm, scratch, part, total;
};

BwdLayout bwd_layout(const tp_attn_s* h, int64_t N, int64_t E) {
  AttnArgs a = h->proto;
  a.N = (int)N;
  a.E = (int)E;
  hist_plan(a);
  window_plan(a);
  BwdLayout L;
  size_t off = 0;
  const size_t e = (size_t)std::max<int64_t>(E, 1);
  L.rec = off;
  off += al256(sizeof(float2) * e * a.H);
  L.dst = off;
  off += al256(sizeof(int32_t) * e);
  L.hist = off;
  off += al256(sizeof(float) * (size_t)a.hist_ctas * a.K * a.H);
  L.colptr = off;
  off += al256(sizeof(int32_t) * (size_t)(N + 1));
  L.perm = off;
  off += al256(sizeof(int32_t) * e);
  L.scratch = off;
  off += al256(sizeof(int32_t) * (size_t)transpose_scratch_ints(N, E));
  L.part = off;              // the receiver pass's and the sender pass's in turn
  off += al256(std::max(part_bytes(a, kRecv), part_bytes(a, kSend)));
  L.total = off;
  return L;
}

tp_status_t attn_sizes(tp_attn_t h, int64_t N, int64_t E) {
  if (!h) return set_failure(TP_ERR_INVALID_ARG, "attention is NULL");
  if (N < 0 || E < 0) return set_failure(TP_ERR_INVALID_ARG, "N and E must be non-negative");
  if (E > 0x7fffffff - (1 << 22) || N * h->proto.H > 0x7fffffff - (1 << 22))
    return set_failure(TP_ERR_UNSUPPORTED, "E and N * heads must stay below 2^31 - 2^22 (int32 indices)");
  return TP_OK;
}

// What forward and backward check alike; fills the inputs of `a`.
tp_status_t attn_inputs(tp_attn_t h, int64_t N, int64_t E, const int32_t* rowptr, const int32_t* src,
                        const int32_t* bucket, const float* q, int64_t ldq, const float* k, int64_t ldk,
                        const float* v, int64_t ldv, const float* table, float scale, double p, const int64_t* rng,
                        int64_t site, AttnArgs& a) {
  a = h->proto;
  if (!rowptr || !q || !k || !v || (E > 0 && !src)) return set_failure(TP_ERR_INVALID_ARG, "NULL input");
  if (ldq < a.dq || ldk < a.dq || ldv < a.dv) return set_failure(TP_ERR_INVALID_ARG, "a row stride is below the row's width");
  if (bucket && a.K == 0) return set_failure(TP_ERR_INVALID_ARG, "buckets given to an attention without buckets");
  if (table && !bucket && E > 0) return set_failure(TP_ERR_INVALID_ARG, "table needs bucket");
  if (table && a.K == 0) return set_failure(TP_ERR_INVALID_ARG, "table given to an attention without buckets");
  if (!std::isfinite(scale)) return set_failure(TP_ERR_INVALID_ARG, "scale must be finite");
  if (!drop_args(p, rng, site, a.drop))
    return set_failure(TP_ERR_INVALID_ARG, "p_drop must lie in [0, 1) and p_drop > 0 needs rng");
  for (const void* t : {(const void*)rowptr, (const void*)src, (const void*)bucket, (const void*)q, (const void*)k,
                        (const void*)v, (const void*)table})
    if (!al4(t)) return set_failure(TP_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(rng) & 7u) return set_failure(TP_ERR_INVALID_ARG, "rng must be 8-byte aligned");
  a.N = (int)N;
  a.E = (int)E;
  a.rowptr = rowptr;
  a.src = src;
  a.bucket = bucket;
  a.q = q;
  a.k = k;
  a.v = v;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.table = table;
  a.scale = scale;
  window_plan(a);
  return TP_OK;
}

bool rows4(const AttnArgs& a) {
  return al16(a.q) && al16(a.k) && al16(a.v) && a.ldq % 4 == 0 && a.ldk % 4 == 0 && a.ldv % 4 == 0;
}

bool head_map(const std::vector<IrrepTerm>& t, int heads, HeadMap& m, int& dim) {
  int64_t off = 0;
  m.nb = 0;
  m.hd = 0;
  for (const IrrepTerm& b : t) {
    if (b.mul % heads != 0) return false;
    m.off[m.nb] = (int)off;
    m.len[m.nb] = b.mul / heads * (2 * b.l + 1);
    m.hd += m.len[m.nb++];
    off += (int64_t)b.mul * (2 * b.l + 1);
  }
  dim = (int)off;
  return true;
}

}  // namespace

extern "C" {

tp_status_t tp_attn_create(tp_attn_t* attn, const char* irreps_qk, const char* irreps_v, int32_t heads,
                           int32_t n_buckets) try {
  if (!attn) return set_failure(TP_ERR_INVALID_ARG, "attention is NULL");
  *attn = nullptr;
  if (heads < 1) return set_failure(TP_ERR_INVALID_ARG, "heads must be positive");
  if (heads > 32) return set_failure(TP_ERR_UNSUPPORTED, "at most 32 heads");
  if (n_buckets < 0) return set_failure(TP_ERR_INVALID_ARG, "n_buckets must be non-negative");
  if (n_buckets > 4096 || n_buckets * heads > 32768)
    return set_failure(TP_ERR_UNSUPPORTED, "at most 4096 buckets and 32768 table entries");
  tp_attn_s h;
  std::memset(&h, 0, sizeof(h));
  h.vec4 = true;
  struct Side {
    const char* irreps;
    const char* name;
    HeadMap* map;
    int* dim;
  };
  for (const Side& side : {Side{irreps_qk, "irreps_qk", &h.proto.mq, &h.proto.dq},
                           Side{irreps_v, "irreps_v", &h.proto.mv, &h.proto.dv}}) {
    std::vector<IrrepTerm> t;
    std::string why;
    if (!parse_irreps_terms(side.irreps, t, why))
      return set_failure(TP_ERR_INVALID_ARG, std::string(side.name) + ": " + why);
    if ((int)t.size() > kAttnMaxBlocks) return set_failure(TP_ERR_UNSUPPORTED, "at most 16 irreps blocks");
    int64_t width = 0;
    for (const IrrepTerm& b : t) {
      if (b.l > 3) return set_failure(TP_ERR_UNSUPPORTED, "l > 3");
      width += (int64_t)b.mul * (2 * b.l + 1);
    }
    if (width > (int64_t)4096 * heads) return set_failure(TP_ERR_UNSUPPORTED, "a head has at most 4096 floats");
    if (!head_map(t, heads, *side.map, *side.dim))
      return set_failure(TP_ERR_INVALID_ARG, std::string(side.name) + ": heads must divide every multiplicity");
    for (int b = 0; b < side.map->nb; ++b) h.vec4 = h.vec4 && side.map->len[b] % 4 == 0;
  }
  h.proto.H = heads;
  h.proto.K = n_buckets;
  *attn = new tp_attn_s(h);
  return TP_OK;
} catch (...) {
  return TP_ERR_INVALID_ARG;   // out of host memory
}

tp_status_t tp_attn_destroy(tp_attn_t attn) {
  delete attn;
  return TP_OK;
}

tp_status_t tp_attn_query(tp_attn_t attn, int64_t* qk_dim, int64_t* v_dim) {
  if (!attn) return set_failure(TP_ERR_INVALID_ARG, "attention is NULL");
  if (qk_dim) *qk_dim = attn->proto.dq;
  if (v_dim) *v_dim = attn->proto.dv;
  return TP_OK;
}

tp_status_t tp_attn_workspace_size(tp_attn_t attn, int64_t N, int64_t E, int32_t op, size_t* bytes) {
  tp_status_t st = attn_sizes(attn, N, E);
  if (st != TP_OK) return st;
  if (!bytes) return set_failure(TP_ERR_INVALID_ARG, "bytes is NULL");
  if (op != TP_OP_FWD && op != TP_OP_BWD) return set_failure(TP_ERR_INVALID_ARG, "op must be TP_OP_FWD or TP_OP_BWD");
  AttnArgs a = attn->proto;
  a.E = (int)E;
  window_plan(a);
  *bytes = op == TP_OP_FWD ? al256(part_bytes(a, kFwd)) : bwd_layout(attn, N, E).total;
  return TP_OK;
}

tp_status_t tp_attn_fwd(tp_attn_t attn, int64_t N, int64_t E, const int32_t* rowptr, const int32_t* src,
                        const int32_t* bucket, const float* q, int64_t ldq, const float* k, int64_t ldk,
                        const float* v, int64_t ldv, const float* table, float scale, double p_drop,
                        const int64_t* rng, int64_t site, float* y, float* lse, void* ws, size_t ws_bytes,
                        tp_stream_t stream) {
  tp_status_t st = attn_sizes(attn, N, E);
  if (st != TP_OK || N == 0) return st;
  AttnArgs a;
  st = attn_inputs(attn, N, E, rowptr, src, bucket, q, ldq, k, ldk, v, ldv, table, scale, p_drop, rng, site, a);
  if (st != TP_OK) return st;
  if (!y) return set_failure(TP_ERR_INVALID_ARG, "y must not be NULL");
  if (!al4(y) || !al4(lse)) return set_failure(TP_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  const size_t need = part_bytes(a, kFwd);
  if (need > 0 && (!ws || ws_bytes < need)) return set_failure(TP_ERR_WORKSPACE, "workspace too small");
  if (need > 0 && (reinterpret_cast<uintptr_t>(ws) & 255u))
    return set_failure(TP_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  a.y = y;
  a.lse = lse;
  return cuda_status(launch_pass(kFwd, a, attn->vec4 && rows4(a) && al16(y), static_cast<float*>(ws), reinterpret_cast<cudaStream_t>(stream)),
                     "tp_attn_fwd");
}

tp_status_t tp_attn_bwd(tp_attn_t attn, int64_t N, int64_t E, const int32_t* rowptr, const int32_t* src,
                        const int32_t* colptr, const int32_t* perm, const int32_t* bucket, const float* q,
                        int64_t ldq, const float* k, int64_t ldk, const float* v, int64_t ldv, const float* table,
                        float scale, double p_drop, const int64_t* rng, int64_t site, const float* y,
                        const float* lse, const float* gy, float* gq, int64_t ldgq, float* gk, int64_t ldgk,
                        float* gv, int64_t ldgv, float* gtable, void* ws, size_t ws_bytes, tp_stream_t stream) {
  tp_status_t st = attn_sizes(attn, N, E);
  if (st != TP_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (gtable && attn->proto.K == 0)
    return set_failure(TP_ERR_INVALID_ARG, "gtable asked of an attention without buckets");
  if (!gq && !gk && !gv && !gtable) return TP_OK;
  if (!al4(gtable)) return set_failure(TP_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  if (N == 0 || E == 0) {
    if (gtable) {
      cudaError_t e = cudaMemsetAsync(gtable, 0, sizeof(float) * (size_t)attn->proto.K * attn->proto.H, s);
      if (e != cudaSuccess) return cuda_status(e, "tp_attn_bwd");
    }
    if (N == 0) return TP_OK;
  }
  AttnArgs a;
  st = attn_inputs(attn, N, E, rowptr, src, bucket, q, ldq, k, ldk, v, ldv, table, scale, p_drop, rng, site, a);
  if (st != TP_OK) return st;
  if (!y || !lse || !gy) return set_failure(TP_ERR_INVALID_ARG, "y, lse and gy must not be NULL");
  if (gtable && !table) return set_failure(TP_ERR_INVALID_ARG, "gtable needs table");
  if ((colptr == nullptr) != (perm == nullptr) && E > 0)
    return set_failure(TP_ERR_INVALID_ARG, "colptr and perm must both be given or both be NULL");
  if ((gq && ldgq < a.dq) || (gk && ldgk < a.dq) || (gv && ldgv < a.dv))
    return set_failure(TP_ERR_INVALID_ARG, "a row stride is below the row's width");
  for (const void* t : {(const void*)colptr, (const void*)perm, (const void*)y, (const void*)lse, (const void*)gy,
                        (const void*)gq, (const void*)gk, (const void*)gv})
    if (!al4(t)) return set_failure(TP_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  const BwdLayout L = bwd_layout(attn, N, E);
  if (!ws || ws_bytes < L.total) return set_failure(TP_ERR_WORKSPACE, "workspace too small");
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return set_failure(TP_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  char* w = static_cast<char*>(ws);
  const bool send = gk || gv;
  cudaError_t e = cudaSuccess;
  if (send && !perm) {
    int32_t* cp = reinterpret_cast<int32_t*>(w + L.colptr);
    int32_t* pm = reinterpret_cast<int32_t*>(w + L.perm);
    e = launch_csr_transpose(a.N, a.E, src, cp, pm, reinterpret_cast<int32_t*>(w + L.scratch), s);
    if (e != cudaSuccess) return cuda_status(e, "transpose");
    colptr = cp;
    perm = pm;
  }
  a.colptr = colptr;
  a.perm = perm;
  a.y_in = y;
  a.lse_in = lse;
  a.gy = gy;
  a.gq = gq;
  a.gk = gk;
  a.gv = gv;
  a.ldgq = ldgq;
  a.ldgk = ldgk;
  a.ldgv = ldgv;
  a.gtable = gtable;
  a.rec = send || gtable ? reinterpret_cast<float2*>(w + L.rec) : nullptr;
  a.dst = reinterpret_cast<int32_t*>(w + L.dst);
  a.hist = reinterpret_cast<float*>(w + L.hist);
  const bool vec4 = attn->vec4 && rows4(a) && al16(y) && al16(gy) && al16(gq) && al16(gk) && al16(gv) &&
                    (!gq || ldgq % 4 == 0) && (!gk || ldgk % 4 == 0) && (!gv || ldgv % 4 == 0);
  float* part = reinterpret_cast<float*>(w + L.part);
  e = launch_pass(kRecv, a, vec4, part, s);
  if (e == cudaSuccess && send) e = launch_pass(kSend, a, vec4, part, s);
  if (e == cudaSuccess && gtable && E > 0) {
    hist_plan(a);
    const size_t smem = sizeof(float) * (size_t)a.K * a.H * a.hist_copies;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(k_attn_table, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) {
      k_attn_table<<<a.hist_ctas, kAttnThreads, smem, s>>>(a);
      count_launches(1);
      e = cudaGetLastError();
    }
    if (e == cudaSuccess && a.hist_ctas > 1) {
      k_attn_table_sum<<<(a.K * a.H + 3) / 4, 128, 0, s>>>(a);
      count_launches(1);
      e = cudaGetLastError();
    }
  }
  return cuda_status(e, "tp_attn_bwd");
}

tp_status_t tp_distance_buckets(int64_t E, const float* vec, int32_t n_bounds, const float* bounds, float cutoff,
                                int32_t* bucket, tp_stream_t stream) {
  if (E < 0 || n_bounds < 0) return set_failure(TP_ERR_INVALID_ARG, "E and n_bounds must be non-negative");
  if (n_bounds > kMaxBounds) return set_failure(TP_ERR_UNSUPPORTED, "at most 1023 bounds");
  if (!(cutoff >= 0.0f)) return set_failure(TP_ERR_INVALID_ARG, "cutoff must be non-negative (+inf for none)");
  if (E == 0) return TP_OK;
  if (E >= (int64_t)1 << 40) return set_failure(TP_ERR_UNSUPPORTED, "E too large");
  if (!vec || !bucket || (n_bounds > 0 && !bounds)) return set_failure(TP_ERR_INVALID_ARG, "NULL input or output");
  if (!al4(vec) || !al4(bounds) || !al4(bucket)) return set_failure(TP_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  const int64_t grid = std::min<int64_t>((E + 255) / 256, 148 * 8);
  k_buckets<<<(unsigned)grid, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(E, vec, n_bounds, bounds,
                                                                              (double)cutoff * (double)cutoff, bucket);
  count_launches(1);
  return cuda_status(cudaGetLastError(), "tp_distance_buckets");
}

}  // extern "C"
