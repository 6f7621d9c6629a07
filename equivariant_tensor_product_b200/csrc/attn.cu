// Equivariant neighbour attention (include/tp_attn.h): softmax over each receiver's edges, with a
// bias per distance bucket and dropout of the probabilities, and its backward pass.
//
// Mapping.  A head's floats (its part of every irreps block) are cut into chunks of V = 4 (2, 1)
// floats and dealt to a group of G lanes, S chunks a lane, so that a lane's chunks of q, of the
// accumulators and of the gathered rows stay in registers and a dot product ends in log2 G
// shuffles.  A warp holds 32 / G heads of one receiver; heads beyond 1,024 floats take a whole
// CTA (WIDE), whose dot products are joined through shared memory.
//
// A warp takes the edges of a receiver 32 at a time.  One lane reads one edge (sender, bucket,
// dropout choices); edges that take no part are struck out and the rest is closed up in shared
// memory.  Forward, per batch: (a) the logits, U edges at a time, each lane's chunks of U rows of k
// in flight at once; (b) the softmax of the batch with one lane per edge and head -- bias, running
// maximum, exp and sum cost a few instructions per edge there, where doing them for every edge in
// every lane of its group cost more than the products; (c) the sum of p v, again U rows at a time.
// The receiver pass of the backward needs no running maximum (p = exp(s - lse)), so it keeps the
// rows of k in registers between the logit and gq and walks the edges once.  The sender pass
// finds (ds, r p) in the workspace and only adds up.
//
// Long rows.  A receiver (sender) of more than `hub` edges would keep one warp busy long after the
// others are done.  Its edges are taken window by window instead: the edge axis is cut into
// windows of win = hub / 2 edges, whose CTAs come before those of the rows.  A window meets at
// most two such rows (the row of its first edge and the row of its last one), finds them by a
// 33-way search in the row pointers and leaves a partial row for each; a join kernel adds a row's
// partials up in window order.  Graphs of at most 320 edges have neither windows nor the join.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>
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
  int row_ctas, win_ctas;    // CTAs of the rows, and of the windows before them
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
  uint32_t ldq, ldk, ldv;    // row strides in bytes
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
  int64_t ldgq, ldgk, ldgv;  // in floats
  float* gtable;
  float2* rec;               // workspace [E][H]: (ds, r p) of the backward pass
  int32_t* dst;              // workspace [E]: receiver, -1 for an edge that takes no part
  float* hist;               // workspace [hist_ctas][K * H]
  int hist_ctas, hist_copies, hist_lanes;
  int table_here;            // sender pass: the table's CTAs come behind it
  int threads;               // of a CTA of the passes, and of the table's, so that its sums do not depend on where it runs
  HeadMap mq, mv;
};

enum Pass { kFwd, kRecv, kSend };

// Rows in flight (U) and CTAs a SM, which holds the registers down, for S chunks a lane.  Both hide the
// latency of the gathers and both want registers; what is first in short supply differs by pass.  Measured
// with 16-byte chunks, 46,080 edges of 288 floats and 3.0M edges of 1,152 floats (S = 3), 162,892 edges of
// 1,024 floats (S = 4):
//   forward  S = 3: U 4 at 4 CTAs 15.8 us / 3.78 ms, U 4 at 5 18.2 / 4.08, U 2 at 5 20.0 / 4.54
//            S = 4: U 2 at 5 CTAs 103 us, U 1 at 6 161
//   receiver S = 3: U 2 at 4 CTAs 17.7 us / 4.07 ms, U 4 at 3 18.0 / 4.85, U 2 at 5 21.3 / 4.80
//            S = 4: U 2 at 4 CTAs 116 us, U 2 at 3 121, U 1 at 5 126
//   sender   S = 3: U 4 at 3 CTAs 16.1 us / 4.28 ms, U 2 at 4 18.4 / 4.21, U 2 at 5 20.1 / 4.01
//            S = 4: U 1 at 5 CTAs 97 us, U 2 at 4 103
// and with 4-byte chunks, 100,003 edges of 189 floats (S = 4): forward U 4 at 5 CTAs 45 us, at 6 49; receiver
// U 2 at 5 47, U 4 at 5 53; sender U 2 at 6 33, at 5 37.
__host__ __device__ constexpr int rows_at_once(Pass pass, int V, int S, bool wide) {
  if (wide) return S <= 4 ? 2 : 1;
  if (V < 4) return S <= 3 || (S == 4 && pass == kFwd) ? 4 : S == 4 || pass != kRecv ? 2 : 1;
  if (S <= 2) return 4;
  if (S == 3) return pass == kRecv ? 2 : 4;
  return S == 4 && pass != kSend ? 2 : 1;
}
__host__ __device__ constexpr int ctas_per_sm(Pass pass, int V, int S) {
  if (S >= 6) return S == 6 ? 3 : 2;
  if (V == 1) return pass == kSend ? 6 : 5;
  if (V == 2) return pass == kRecv ? 4 : 5;
  if (S <= 2) return 4;
  if (S == 3) return pass == kSend ? 3 : 4;
  return pass == kRecv ? 4 : 5;
}

constexpr int kMinWindow = 64, kFewWindows = 160;

// The kernels of one call follow each other by programmatic dependent launch: a kernel lets the next
// one be set up from its start on, and the next one waits here, before it touches anything that an
// earlier one writes, until all of them are done.
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
__device__ __forceinline__ Vec<V> zero_vec() {
  Vec<V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.x[i] = 0.0f;
  return r;
}

// Reads a chunk.  GUARD: a lane without one (on = false) gets zeros.
template <int V, bool GUARD>
__device__ __forceinline__ Vec<V> load_vec(const char* p, bool on) {
  Vec<V> r;
  if constexpr (GUARD) r = zero_vec<V>();
  if (!GUARD || on) {
    if constexpr (V == 4) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(p));
      r.x[0] = t.x, r.x[1] = t.y, r.x[2] = t.z, r.x[3] = t.w;
    } else if constexpr (V == 2) {
      const float2 t = __ldg(reinterpret_cast<const float2*>(p));
      r.x[0] = t.x, r.x[1] = t.y;
    } else {
      r.x[0] = __ldg(reinterpret_cast<const float*>(p));
    }
  }
  return r;
}

// Byte address of row j: one 32 x 32 -> 64 bit multiply-add.  A lane's chunks lie at 32-bit offsets from it.
__device__ __forceinline__ const char* row_at(const float* p, int j, uint32_t row_bytes) {
  return reinterpret_cast<const char*>(p) + (uint64_t)(uint32_t)j * row_bytes;
}

template <int V>
__device__ __forceinline__ void store_vec(float* p, const Vec<V>& r) {
  if constexpr (V == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(r.x[0], r.x[1], r.x[2], r.x[3]);
  } else if constexpr (V == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(r.x[0], r.x[1]);
  } else {
    *p = r.x[0];
  }
}

__device__ __forceinline__ float exp_of(float x) { return exp2f(x * kLog2e); }

__device__ __forceinline__ int clamp_edge(int e, int E) { return min(max(e, 0), E); }

// The rows r of `ptr` with ptr[r] <= e < ptr[r + 1], or -1, for two edges e: 32 probes a step, both
// searches at once; the same answers in every lane.
__device__ __forceinline__ void find_rows(const int32_t* __restrict__ ptr, int N, int e0, int e1, int& r0, int& r1) {
  const int from = __ldg(ptr), to = __ldg(ptr + N), lane = threadIdx.x & 31;
  int lo[2] = {0, 0}, hi[2] = {N, N};
  const int e[2] = {e0, e1};
  while (hi[0] - lo[0] > 1 || hi[1] - lo[1] > 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int step = max((hi[i] - lo[i] + 32) / 33, 1);
      const int64_t pos = lo[i] + (int64_t)(lane + 1) * step;
      const int below = __popc(__ballot_sync(kFull, pos < hi[i] && __ldg(ptr + min(pos, (int64_t)hi[i])) <= e[i]));
      lo[i] += below * step;
      hi[i] = min(hi[i], lo[i] + step);
    }
  }
  r0 = e0 >= from && e0 < to ? lo[0] : -1;
  r1 = e1 >= from && e1 < to ? lo[1] : -1;
}

// A stretch of one row's edges that a CTA's warps work on: a whole row, or a window's share of a long one.
struct Task {
  int row, head0, split, W, lo, hi;
  float* part;               // where a window leaves its partial row
  bool write;                // false: a long row, which the windows deal with
};

// The tasks of this CTA.  Rows: one.  Windows: the heads of up to two long rows, found here.  Where a row has
// one warp, a CTA has no more: with four rows a CTA the warps of the three shorter ones stood idle until
// the longest was done (1.18M edges with degrees up to 150: 366 us, against 263 with equal degrees).
template <bool WIDE>
struct Tasks {
  int n, next, window, head_first, row0, row1;

  __device__ __forceinline__ Tasks(const AttnArgs& a, const int32_t* __restrict__ ptr) {
    next = 0;
    n = 1;
    if ((int)blockIdx.x >= a.win_ctas) return;
    window = blockIdx.x;
    head_first = 0;
    int groups = WIDE ? a.H : a.groups;
    if (!WIDE && a.W == 1) {             // one head group
      head_first = window % groups * a.hw;
      window /= groups;
      groups = 1;
    }
    const int first = window * a.win;
    find_rows(ptr, a.N, first, min(first + a.win, a.E) - 1, row0, row1);
    if (row0 >= 0 && __ldg(ptr + row0 + 1) - __ldg(ptr + row0) <= a.hub) row0 = -1;
    if (row1 >= 0 && (__ldg(ptr + row1 + 1) - __ldg(ptr + row1) <= a.hub || __ldg(ptr + row1) <= first)) row1 = -1;
    n = row0 < 0 && row1 < 0 ? 0 : 2 * groups;
  }

  __device__ __forceinline__ bool get(const AttnArgs& a, const int32_t* __restrict__ ptr, Task& t) {
    const int warp = threadIdx.x >> 5;
    if (next >= n) return false;
    t.part = nullptr;
    t.write = false;
    t.lo = t.hi = t.split = 0;
    t.W = 1;
    if ((int)blockIdx.x >= a.win_ctas) {
      const int cta = (int)blockIdx.x - a.win_ctas;
      next = 1;
      if (WIDE) {
        t.row = cta / a.H;
        t.head0 = cta - t.row * a.H;
      } else {
        // one head group after the other: what a group reads of k and v stays in L2 for longer
        const int blocks = a.row_ctas / a.groups, g = cta / blocks;
        t.head0 = g * a.hw;
        t.W = a.W;
        t.split = warp % a.W;
        t.row = (cta - g * blocks) * ((int)(blockDim.x >> 5) / a.W) + warp / a.W;
        if (t.row >= a.N) return true;
      }
      t.lo = clamp_edge(__ldg(ptr + t.row), a.E);
      t.hi = clamp_edge(__ldg(ptr + t.row + 1), a.E);
      t.write = a.n_win == 0 || t.hi - t.lo <= a.hub;
      if (!t.write) t.hi = t.lo;
    } else {
      const int per = n / 2, slot = next / per, first = window * a.win;
      if (next > 0) __syncthreads();     // the join buffer is free again
      t.row = slot ? row1 : row0;
      t.head0 = head_first + (next - slot * per) * (WIDE ? 1 : a.hw);
      ++next;
      if (t.row < 0) return true;
      t.write = true;
      t.part = a.part + ((int64_t)window * 2 + slot) * a.part_len;
      t.lo = max(__ldg(ptr + t.row), first);
      t.hi = min(min(__ldg(ptr + t.row + 1), first + a.win), a.E);
      if (!WIDE) {
        t.W = blockDim.x >> 5;
        t.split = warp;
      }
    }
    if (t.W > 1 && t.hi > t.lo) {
      const int per = (t.hi - t.lo + t.W - 1) / t.W;
      t.lo += min(t.split * per, t.hi - t.lo);
      t.hi = min(t.hi, t.lo + per);
    }
    return true;
  }
};

// Which head of the task's row a thread holds, and its chunks: number s G + gl of the head's chunks.
// Lanes beyond the last head shadow it; `live` keeps what they find out of every output.
template <int V, bool WIDE>
struct Lane {
  int h, G, gl, sub;
  bool live;                 // a head of its own, of a row that is this task's to write

  __device__ __forceinline__ Lane(const AttnArgs& a) : h(-1), live(false) {
    const int lane = threadIdx.x & 31;
    G = WIDE ? blockDim.x : 32 / a.hw;
    sub = WIDE ? 0 : lane / G;
    gl = WIDE ? threadIdx.x : lane & (G - 1);
  }
  // Takes up a task; true if the head is another one than before.
  __device__ __forceinline__ bool take(const AttnArgs& a, const Task& t) {
    const int want = t.head0 + sub, was = h;
    h = min(want, a.H - 1);
    live = t.write && want < a.H;
    return __any_sync(kFull, h != was);
  }

  __device__ __forceinline__ bool has(const HeadMap& m, int s) const { return (s * G + gl) * V < m.hd; }
  // Byte offsets of the chunks in a row; a chunk the lane lacks is given the row's first.
  template <int S>
  __device__ __forceinline__ void offsets(const HeadMap& m, uint32_t (&o)[S]) const {
#pragma unroll
    for (int s = 0; s < S; ++s) o[s] = 4u * max(slot_offset(m, h, (s * G + gl) * V), 0);
  }

  // The lane's part in a batch of 32 edges x the warp's heads: entries lane' + 32 i of [edge][head].
  __device__ __forceinline__ int step() const { return WIDE ? 32 : G; }
  __device__ __forceinline__ int first() const { return WIDE ? (int)(threadIdx.x & 31) : gl; }

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

// A warp's place in shared memory for a batch: the live edges' rows, two more words of each, and two
// floats per edge and head.
struct Batch {
  int* row;
  int* b;
  uint32_t* c;
  float* f;                  // [32][hw] floats, or float2
};

__device__ __forceinline__ Batch batch_of_warp(int hw) {
  extern __shared__ __align__(16) unsigned char dyn[];
  int* p = reinterpret_cast<int*>(dyn) + (threadIdx.x >> 5) * (96 + 64 * hw);
  return Batch{p, p + 32, reinterpret_cast<uint32_t*>(p + 64), reinterpret_cast<float*>(p + 96)};
}
// Behind the warps' batches: where the warps of a row, or of a WIDE row's dot products, meet.
__device__ __forceinline__ float* join_of_cta(int hw) {
  extern __shared__ __align__(16) unsigned char dyn[];
  return reinterpret_cast<float*>(dyn) + (blockDim.x >> 5) * (96 + 64 * hw);
}
// Floats of it for a pass: two turns of the dot products, or a warp's partial row for every warp.
constexpr int join_floats(Pass pass, int V, int SQ, int SV, bool wide, int u) {
  if (wide) return pass == kSend ? 0 : 2 * (kAttnWideThreads / 32) * (pass == kRecv ? 2 : 1) * u;
  return kAttnWarps * 32 * (pass == kFwd ? V * SV + 2 : pass == kRecv ? V * SQ : V * (SQ + SV));
}
size_t batch_bytes(int threads, int hw) { return (size_t)(threads / 32) * (96 + 64 * hw) * 4; }

// An entry whose table value is -inf: its edge takes no part for that head, and no row of it may reach
// a sum, whatever it holds.  Such an entry is marked with -0, which no probability is.
__device__ __forceinline__ bool marked(float p) { return __float_as_uint(p) == 0x80000000u; }

template <int V, int SQ, int SV, bool LOOSE, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kAttnWideThreads : kAttnThreads, WIDE ? 1 : ctas_per_sm(kFwd, V, SV)) k_attn_fwd(const __grid_constant__ AttnArgs a) {
  constexpr int U = rows_at_once(kFwd, V, SV, WIDE);
  // rows of k at a time: more where a lane holds but one chunk of them
  constexpr int UA = WIDE ? U : SQ == 1 || (SQ == 2 && V < 4) ? 8 : SQ == 2 ? 4 : U;
  float* const join = join_of_cta(a.hw);
  let_next_launch();
  const int lane = threadIdx.x & 31;
  const Batch B = batch_of_warp(a.hw);
  int turn = 0;
  DropKey key{};
  if (a.drop.rng) key = drop_key(a.drop);
  Tasks<WIDE> tasks(a, a.rowptr);
  Lane<V, WIDE> L(a);
  uint32_t oq[SQ], ov[SV];
  for (Task t; tasks.get(a, a.rowptr, t);) {
    Vec<V> q[SQ], acc[SV];
    float m = -INFINITY, l = 0.0f;       // maximum of the group's logits; the lane's share of the sum
    if (L.take(a, t)) {
      L.offsets(a.mq, oq);
      L.offsets(a.mv, ov);
    }
    const char* q_row = row_at(a.q, t.row, a.ldq);
#pragma unroll
    for (int s = 0; s < SQ; ++s)
      q[s] = load_vec<V, true>(q_row + oq[s], L.live && L.has(a.mq, s));
#pragma unroll
    for (int s = 0; s < SV; ++s) acc[s] = zero_vec<V>();
    for (int base = t.lo; base < t.hi; base += 32) {
      const EdgeLane mine = read_edge(a, key, base + lane, base + lane < t.hi, t.head0, a.hw);
      const uint32_t live = __ballot_sync(kFull, mine.j >= 0);
      const int n = __popc(live);
      if (n == 0) continue;
      __syncwarp();
      if (mine.j >= 0) {
        const int at = __popc(live & ((1u << lane) - 1u));
        B.row[at] = mine.j;
        B.b[at] = mine.b;
        B.c[at] = mine.keep;
      }
      __syncwarp();
      // (a) logits.  The last round repeats the last edge where there are fewer left.
      for (int t0 = 0; t0 < n; t0 += UA) {
        float dot[UA];
        Vec<V> x[UA][SQ];
#pragma unroll
        for (int u = 0; u < UA; ++u) {
          const char* row = row_at(a.k, B.row[min(t0 + u, n - 1)], a.ldk);
#pragma unroll
          for (int s = 0; s < SQ; ++s)
            x[u][s] = s < SQ - 1 && !LOOSE ? load_vec<V, false>(row + oq[s], true)
                                           : load_vec<V, true>(row + oq[s], L.has(a.mq, s));
        }
#pragma unroll
        for (int u = 0; u < UA; ++u) {
          dot[u] = 0.0f;
#pragma unroll
          for (int s = 0; s < SQ; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) dot[u] = fmaf(q[s].x[i], x[u][s].x[i], dot[u]);
        }
        L.sum(dot, join, turn);
        if (L.first() == 0) {
#pragma unroll
          for (int u = 0; u < UA; ++u) B.f[min(t0 + u, n - 1) * a.hw + L.sub] = dot[u];
        }
      }
      __syncwarp();
      // (b) softmax of the batch
      float top = m;
      bool any_out = false;
      for (int i = L.first(); i < n; i += L.step()) {
        float& f = B.f[i * a.hw + L.sub];
        const float bias = a.table && L.live ? __ldg(a.table + (int64_t)B.b[i] * a.H + L.h) : 0.0f;
        const bool out = bias == -INFINITY;
        any_out |= out;
        f = out ? -INFINITY : fmaf(f, a.scale, bias);
        top = fmaxf(top, f);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (L.step() > o) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      const float ref = top == -INFINITY ? 0.0f : top;
      const float shrink = exp_of(m - ref);
      m = top;
      l *= shrink;
#pragma unroll
      for (int s = 0; s < SV; ++s)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[s].x[i] *= shrink;
      for (int i = L.first(); i < n; i += L.step()) {
        float& f = B.f[i * a.hw + L.sub];
        const bool out = any_out && f == -INFINITY;
        const float p = exp_of(f - ref);
        l += p;
        f = out ? -0.0f : (B.c[i] >> L.sub) & 1u ? p : 0.0f;
      }
      any_out = __any_sync(kFull, any_out);
      __syncwarp();
      // (c) sum of p v
      for (int t0 = 0; t0 < n; t0 += U) {
        Vec<V> x[U][SV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const char* row = row_at(a.v, B.row[min(t0 + u, n - 1)], a.ldv);
#pragma unroll
          for (int s = 0; s < SV; ++s)
            x[u][s] = s < SV - 1 && !LOOSE ? load_vec<V, false>(row + ov[s], true)
                                           : load_vec<V, true>(row + ov[s], L.has(a.mv, s));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (t0 + u >= n) break;
          const float p = B.f[(t0 + u) * a.hw + L.sub];
          if (any_out && marked(p)) continue;
#pragma unroll
          for (int s = 0; s < SV; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[s].x[i] = fmaf(p, x[u][s].x[i], acc[s].x[i]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (L.step() > o) l += __shfl_xor_sync(kFull, l, o);
    if constexpr (!WIDE) {
      if (t.W > 1) {                       // join the warps of a row in order
        const int warp = threadIdx.x >> 5;
        float* mine = join + warp * (V * SV + 2) * 32;
        if (t.split > 0) {
          mine[lane] = m;
          mine[32 + lane] = l;
#pragma unroll
          for (int s = 0; s < SV; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) mine[(2 + s * V + i) * 32 + lane] = acc[s].x[i];
        }
        __syncthreads();
        for (int w = 1; t.split == 0 && w < t.W; ++w) {
          const float* other = join + (warp + w) * (V * SV + 2) * 32;
          const float m2 = other[lane], top = fmaxf(m, m2), ref = top == -INFINITY ? 0.0f : top;
          const float f1 = exp_of(m - ref), f2 = exp_of(m2 - ref);
          l = l * f1 + other[32 + lane] * f2;
#pragma unroll
          for (int s = 0; s < SV; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[s].x[i] = acc[s].x[i] * f1 + other[(2 + s * V + i) * 32 + lane] * f2;
          m = top;
        }
      }
    }
    if (L.live && t.split == 0) {
      if (t.part) {
#pragma unroll
        for (int s = 0; s < SV; ++s)
          if (L.has(a.mv, s)) store_vec<V>(t.part + ov[s] / 4, acc[s]);
        if (L.gl == 0) {
          t.part[a.part_len - 2 * a.H + L.h] = m;
          t.part[a.part_len - a.H + L.h] = l;
        }
      } else {
        const bool none = m == -INFINITY && l == 0.0f;
        const float f = none ? 0.0f : a.drop.inv_keep / l;
#pragma unroll
        for (int s = 0; s < SV; ++s) {
          if (!L.has(a.mv, s)) continue;
#pragma unroll
          for (int i = 0; i < V; ++i) acc[s].x[i] *= f;
          store_vec<V>(a.y + (int64_t)t.row * a.dv + ov[s] / 4, acc[s]);
        }
        if (a.lse && L.gl == 0) a.lse[(int64_t)t.row * a.H + L.h] = none ? -INFINITY : m + logf(l);
      }
    }
  }
}

// A row whose log-sum lies far from zero (a constant bias, a mask of the lowest float on every edge) has lost in
// the rounding of lse = m + log l what normalises it: half a unit in the last place is 6e-5 at 2^10, the whole of
// log l from 2^24 on, and exp(s - lse) would be off by as much.  Such rows get the maximum and the sum of their
// exponentials again, from one more sweep over the whole row's rows of k by every task of the row: rare enough
// for a sweep that every window of a long row repeats.  Rows that are not far pay one subtraction an edge
// (whole step: 46,080 edges 53.0 -> 53.2 us, 165,448 edges of 320 floats 725 -> 733).
constexpr float kFarLse = 1024.0f;
__device__ __forceinline__ bool far_from_zero(float lse) { return fabsf(lse) >= kFarLse && fabsf(lse) < INFINITY; }

template <int V, int SQ, int N, bool WIDE>
__device__ __forceinline__ void row_statistics(const AttnArgs& a, const Lane<V, WIDE>& L, int row, const Vec<V> (&q)[SQ],
                                               const uint32_t (&oq)[SQ], float* join, int& turn, float& top, float& l) {
  const int lo = clamp_edge(__ldg(a.rowptr + row), a.E), hi = clamp_edge(__ldg(a.rowptr + row + 1), a.E);
  for (int e0 = lo; e0 < hi; e0 += N) {
    float dot[N], bias[N];                 // bias -inf: takes no part
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int e = min(e0 + u, hi - 1), j = __ldg(a.src + e), b = a.bucket ? __ldg(a.bucket + e) : 0;
      const bool on = e0 + u < hi && (unsigned)j < (unsigned)a.N && (!a.bucket || (unsigned)b < (unsigned)a.K);
      bias[u] = !on ? -INFINITY : a.table && L.live ? __ldg(a.table + (int64_t)b * a.H + L.h) : 0.0f;
      dot[u] = 0.0f;
      const char* k_row = row_at(a.k, on ? j : 0, a.ldk);
#pragma unroll
      for (int s = 0; s < SQ; ++s) {
        const Vec<V> x = load_vec<V, true>(k_row + oq[s], on && L.has(a.mq, s));
#pragma unroll
        for (int i = 0; i < V; ++i) dot[u] = fmaf(q[s].x[i], x.x[i], dot[u]);
      }
    }
    L.sum(dot, join, turn);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (bias[u] == -INFINITY) continue;
      const float s = fmaf(dot[u], a.scale, bias[u]), high = fmaxf(top, s);
      l = l * exp_of(top - high) + exp_of(s - high);
      top = high;
    }
  }
}

// Backward, receiver order: gq, and for the sender pass and gtable (ds, r p) of every live edge and head
// and the receiver of every edge.
template <int V, int SQ, int SV, bool LOOSE, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kAttnWideThreads : kAttnThreads, WIDE ? 1 : ctas_per_sm(kRecv, V, SV)) k_attn_bwd_recv(const __grid_constant__ AttnArgs a) {
  constexpr int U = rows_at_once(kRecv, V, SV, WIDE);
  float* const join = join_of_cta(a.hw);
  let_next_launch();
  const int lane = threadIdx.x & 31;
  const Batch B = batch_of_warp(a.hw);
  float2* const w2 = reinterpret_cast<float2*>(B.f);
  int turn = 0;
  DropKey key{};
  if (a.drop.rng) key = drop_key(a.drop);
  Tasks<WIDE> tasks(a, a.rowptr);
  Lane<V, WIDE> L(a);
  uint32_t oq[SQ], ov[SV];
  for (Task t; tasks.get(a, a.rowptr, t);) {
    Vec<V> q[SQ], gy[SV], acc[SQ];
    float delta[2 * U];
#pragma unroll
    for (int u = 0; u < 2 * U; ++u) delta[u] = 0.0f;
    if (L.take(a, t)) {
      L.offsets(a.mq, oq);
      L.offsets(a.mv, ov);
    }
    const char *q_row = row_at(a.q, t.row, a.ldq), *gy_row = row_at(a.gy, t.row, a.dv * 4u), *y_row = row_at(a.y_in, t.row, a.dv * 4u);
#pragma unroll
    for (int s = 0; s < SQ; ++s) {
      q[s] = load_vec<V, true>(q_row + oq[s], L.live && L.has(a.mq, s));
      acc[s] = zero_vec<V>();
    }
#pragma unroll
    for (int s = 0; s < SV; ++s) {
      const bool on = L.live && L.has(a.mv, s);
      gy[s] = load_vec<V, true>(gy_row + ov[s], on);
      const Vec<V> y = load_vec<V, true>(y_row + ov[s], on);
#pragma unroll
      for (int i = 0; i < V; ++i) delta[0] = fmaf(gy[s].x[i], y.x[i], delta[0]);
    }
    L.sum(delta, join, turn);
    float del = delta[0];
    // p = w exp((s - less) - shift): less = lse, or shift = the maximum and w = 1 / the sum where the row is far
    float less = L.live ? __ldg(a.lse_in + (int64_t)t.row * a.H + L.h) : 0.0f, shift = 0.0f, kept = a.drop.inv_keep;
    if (__any_sync(kFull, far_from_zero(less))) {
      float top = -INFINITY, l = 0.0f;
      row_statistics<V, SQ, WIDE ? 2 * U : 2, WIDE>(a, L, t.row, q, oq, join, turn, top, l);
      if (far_from_zero(less) && l > 0.0f) {
        less = 0.0f;
        shift = top;
        kept /= l;
        del /= l;
      }
    }
    for (int base = t.lo; base < t.hi; base += 32) {
      const EdgeLane mine = read_edge(a, key, base + lane, base + lane < t.hi, t.head0, a.hw);
      if (a.rec && base + lane < t.hi && t.head0 == 0 && (!WIDE || threadIdx.x < 32))
        a.dst[base + lane] = mine.j >= 0 ? t.row : -1;
      const uint32_t live = __ballot_sync(kFull, mine.j >= 0);
      const int n = __popc(live);
      if (n == 0) continue;
      __syncwarp();
      const int at = __popc(live & ((1u << lane) - 1u));
      if (mine.j >= 0) {
        B.row[at] = mine.j;
        B.b[at] = mine.b;
        B.c[at] = mine.keep;
      }
      __syncwarp();
      bool any_out = false;              // bias and dropout factor, one lane per edge and head
      for (int i0 = L.first(); i0 < n; i0 += 4 * L.step()) {
        float bias[4];                   // four reads at a time
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + k * L.step();
          bias[k] = a.table && L.live && i < n ? __ldg(a.table + (int64_t)B.b[i] * a.H + L.h) : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + k * L.step();
          if (i >= n) break;
          const bool out = bias[k] == -INFINITY || less == -INFINITY;
          any_out |= out;
          w2[i * a.hw + L.sub] = make_float2(out ? -INFINITY : bias[k] - less, (B.c[i] >> L.sub) & 1u ? kept : 0.0f);
        }
      }
      any_out = __any_sync(kFull, any_out);
      __syncwarp();
      if (mine.j >= 0) B.b[at] = base + lane;
      for (int t0 = 0; t0 < n; t0 += U) {
        float dot[2 * U];
        Vec<V> kk[U][SQ], vv[U][SV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = B.row[min(t0 + u, n - 1)];
          const char *k_row = row_at(a.k, j, a.ldk), *v_row = row_at(a.v, j, a.ldv);
#pragma unroll
          for (int s = 0; s < SQ; ++s)
            kk[u][s] = s < SQ - 1 && !LOOSE ? load_vec<V, false>(k_row + oq[s], true)
                                            : load_vec<V, true>(k_row + oq[s], L.has(a.mq, s));
#pragma unroll
          for (int s = 0; s < SV; ++s)
            vv[u][s] = s < SV - 1 && !LOOSE ? load_vec<V, false>(v_row + ov[s], true)
                                            : load_vec<V, true>(v_row + ov[s], L.has(a.mv, s));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          dot[u] = dot[U + u] = 0.0f;
#pragma unroll
          for (int s = 0; s < SQ; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) dot[u] = fmaf(q[s].x[i], kk[u][s].x[i], dot[u]);
#pragma unroll
          for (int s = 0; s < SV; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) dot[U + u] = fmaf(gy[s].x[i], vv[u][s].x[i], dot[U + u]);
        }
        L.sum(dot, join, turn);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (t0 + u >= n) break;
          float2& w = w2[(t0 + u) * a.hw + L.sub];
          const bool out = any_out && w.x == -INFINITY;
          const float p = out ? 0.0f : exp_of(fmaf(dot[u], a.scale, w.x) - shift);
          const float pr = p * w.y, ds = out ? 0.0f : fmaf(pr, dot[U + u], -p * del);
          __syncwarp();
          if (L.first() == 0) w = make_float2(ds, out ? -0.0f : pr);
          if (out) continue;
#pragma unroll
          for (int s = 0; s < SQ; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[s].x[i] = fmaf(ds, kk[u][s].x[i], acc[s].x[i]);
        }
      }
      __syncwarp();
      if (a.rec && L.live && (!WIDE || threadIdx.x < 32)) {
        for (int i = L.first(); i < n; i += L.step()) {
          a.rec[(int64_t)B.b[i] * a.H + L.h] = w2[i * a.hw + L.sub];
        }
      }
    }
    if constexpr (!WIDE) {
      if (t.W > 1) {
        const int warp = threadIdx.x >> 5;
        if (t.split > 0) {
#pragma unroll
          for (int s = 0; s < SQ; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) join[(warp * SQ * V + s * V + i) * 32 + lane] = acc[s].x[i];
        }
        __syncthreads();
        for (int w = 1; t.split == 0 && w < t.W; ++w)
#pragma unroll
          for (int s = 0; s < SQ; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[s].x[i] += join[((warp + w) * SQ * V + s * V + i) * 32 + lane];
      }
    }
    if (L.live && t.split == 0 && a.gq) {
#pragma unroll
      for (int s = 0; s < SQ; ++s) {
        if (!L.has(a.mq, s)) continue;
        if (t.part) {
          store_vec<V>(t.part + oq[s] / 4, acc[s]);
          continue;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) acc[s].x[i] *= a.scale;
        store_vec<V>(a.gq + (int64_t)t.row * a.ldgq + oq[s] / 4, acc[s]);
      }
    }
  }
}

// gtable[b, h] = sum of ds over the edges of bucket b.  The edges are cut into contiguous ranges, one
// for each group of lanes; a group's lanes own one head each and add into the group's own copy of the
// table in shared memory, edge after edge, so every sum has a fixed order.  The reads of eight edges
// are in flight before the first is added: with one at a time the three latencies of each edge were
// all of the kernel (46,080 edges: 12 us).
__device__ __forceinline__ void table_part(const AttnArgs& a, int cta) {
  extern __shared__ __align__(16) unsigned char dyn[];
  float* copies = reinterpret_cast<float*>(dyn);
  const int KH = a.K * a.H, group = threadIdx.x / a.hist_lanes, h = threadIdx.x % a.hist_lanes;
  for (int i = threadIdx.x; i < KH * a.hist_copies; i += blockDim.x) copies[i] = 0.0f;
  __syncthreads();
  const int lo = max(0, min(__ldg(a.rowptr), a.E)), hi = max(lo, min(__ldg(a.rowptr + a.N), a.E));
  if (group < a.hist_copies && h < a.H) {
    const int64_t ranges = (int64_t)a.hist_ctas * a.hist_copies, r = (int64_t)cta * a.hist_copies + group;
    const int first = lo + (int)((hi - lo) * r / ranges), last = lo + (int)((hi - lo) * (r + 1) / ranges);
    float* mine = copies + group * KH + h;
    constexpr int kAhead = 8;
    for (int e0 = first; e0 < last; e0 += kAhead) {
      int b[kAhead], d[kAhead];
      float ds[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int e = min(e0 + i, last - 1);
        d[i] = a.dst[e];
        b[i] = __ldg(a.bucket + e);
        ds[i] = a.rec[(int64_t)e * a.H + h].x;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (d[i] >= 0 && (unsigned)b[i] < (unsigned)a.K && e0 + i < last) mine[b[i] * a.H] += ds[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < KH; i += blockDim.x) {
    float t = 0.0f;
    for (int c = 0; c < a.hist_copies; ++c) t += copies[c * KH + i];
    (a.hist_ctas == 1 ? a.gtable : a.hist + (int64_t)cta * KH)[i] = t;
  }
}

__global__ void __launch_bounds__(kAttnWideThreads) k_attn_table(const __grid_constant__ AttnArgs a) {
  let_next_launch();
  table_part(a, blockIdx.x);
}

// Tables that leave a CTA few copies: one copy a CTA instead, whose buckets the lane groups share out (bucket b
// belongs to group b mod G), so that an entry still has one thread, which adds its edges in order.  A tile of
// edges is staged in shared memory; each warp looks through it 32 edges at a time, each group picks its own.
// With the groups of table_part, 8,192 entries left one group of eight lanes to walk a CTA's 4,096 edges one
// after another (46,080 edges, 8 heads, 1,024 buckets: 271 us of a backward pass of 310, now 23 of 62).  A CTA
// has up to as many edges as there are buckets (256 at least, more from 296 CTAs on), and they may all be of one
// bucket: chains of thousands of 32-bit additions, of values of both signs.
constexpr int kTableThreads = 512, kTableTile = 256;

__global__ void __launch_bounds__(kTableThreads) k_attn_large_table(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  const int KH = a.K * a.H, lanes = a.hist_lanes;
  float* const table = reinterpret_cast<float*>(dyn);
  float* const ds = table + KH;                                    // [tile][H]
  int* const keys = reinterpret_cast<int*>(ds + kTableTile * a.H); // [tile]: bucket, -1 for an edge that takes no part
  let_next_launch();
  for (int i = threadIdx.x; i < KH; i += kTableThreads) table[i] = 0.0f;
  const int lo = max(0, min(__ldg(a.rowptr), a.E)), hi = max(lo, min(__ldg(a.rowptr + a.N), a.E));
  const int first = lo + (int)((int64_t)(hi - lo) * blockIdx.x / a.hist_ctas);
  const int last = lo + (int)((int64_t)(hi - lo) * (blockIdx.x + 1) / a.hist_ctas);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = 32 / lanes, groups = kTableThreads / lanes;
  const int mine = lane / lanes, h = lane & (lanes - 1);
  for (int e0 = first; e0 < last; e0 += kTableTile) {
    const int n = min(kTableTile, last - e0);
    __syncthreads();
    for (int i = threadIdx.x; i < kTableTile; i += kTableThreads) {
      const int b = i < n && a.dst[e0 + i] >= 0 ? __ldg(a.bucket + e0 + i) : -1;
      keys[i] = (unsigned)b < (unsigned)a.K ? b : -1;
    }
    for (int i = threadIdx.x; i < n * a.H; i += kTableThreads) ds[i] = a.rec[(int64_t)e0 * a.H + i].x;
    __syncthreads();
    for (int j = 0; j < n; j += 32) {
      const int key = keys[j + lane], owner = key < 0 ? -1 : key & (groups - 1);
      if (__ballot_sync(kFull, owner >= 0 && owner / per == warp) == 0) continue;
      unsigned todo = 0;
      for (int g = 0; g < per; ++g) {
        const unsigned of_g = __ballot_sync(kFull, owner == warp * per + g);
        if (g == mine) todo = of_g;
      }
      for (; todo != 0; todo &= todo - 1) {
        const int i = j + __ffs(todo) - 1;
        if (h < a.H) table[keys[i] * a.H + h] += ds[i * a.H + h];
      }
      __syncwarp();
    }
  }
  __syncthreads();
  float* const out = a.hist_ctas == 1 ? a.gtable : a.hist + (int64_t)blockIdx.x * KH;
  for (int i = threadIdx.x; i < KH; i += kTableThreads) out[i] = table[i];
}

// One warp per entry of gtable: the CTAs' partials in a fixed order, in 64 bits (up to 1,184 terms of both
// signs).
__device__ __forceinline__ void table_sum(const AttnArgs& a, int o) {
  const int KH = a.K * a.H, lane = threadIdx.x & 31;
  if (o >= KH) return;
  double t = 0.0;
#pragma unroll 4
  for (int c = lane; c < a.hist_ctas; c += 32) t += (double)a.hist[(int64_t)c * KH + o];
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) t += __shfl_xor_sync(kFull, t, s);
  if (lane == 0) a.gtable[o] = (float)t;
}

// Backward, sender order: gk[j] = scale sum ds q[i], gv[j] = sum r p gy[i] over the edges that leave j.
template <int V, int SQ, int SV, bool LOOSE, bool WIDE>
__global__ void __launch_bounds__(WIDE ? kAttnWideThreads : kAttnThreads, WIDE ? 1 : ctas_per_sm(kSend, V, SV)) k_attn_bwd_send(const __grid_constant__ AttnArgs a) {
  constexpr int U = rows_at_once(kSend, V, SV, WIDE);
  float* const join = join_of_cta(a.hw);
  let_next_launch();
  if ((int)blockIdx.x >= a.row_ctas + a.win_ctas) {
    wait_for_previous();
    table_part(a, (int)blockIdx.x - a.row_ctas - a.win_ctas);
    return;
  }
  const int lane = threadIdx.x & 31;
  const Batch B = batch_of_warp(a.hw);
  float2* const w2 = reinterpret_cast<float2*>(B.f);
  const int e_lo = max(__ldg(a.rowptr), 0), e_hi = min(__ldg(a.rowptr + a.N), a.E);
  Tasks<WIDE> tasks(a, a.colptr);
  wait_for_previous();
  Lane<V, WIDE> L(a);
  uint32_t oq[SQ], ov[SV];
  for (Task t; tasks.get(a, a.colptr, t);) {
    Vec<V> ak[SQ], av[SV];
    if (L.take(a, t)) {
      L.offsets(a.mq, oq);
      L.offsets(a.mv, ov);
    }
#pragma unroll
    for (int s = 0; s < SQ; ++s) ak[s] = zero_vec<V>();
#pragma unroll
    for (int s = 0; s < SV; ++s) av[s] = zero_vec<V>();
    for (int base = t.lo; base < t.hi; base += 32) {
      int e = -1, i = -1;
      if (base + lane < t.hi) {
        e = __ldg(a.perm + base + lane);
        if (e >= e_lo && e < e_hi) i = a.dst[e];
        if (i >= a.N) i = -1;              // an edge that no row of the row pointers held
      }
      const uint32_t live = __ballot_sync(kFull, i >= 0);
      const int n = __popc(live);
      if (n == 0) continue;
      __syncwarp();
      if (i >= 0) {
        const int at = __popc(live & ((1u << lane) - 1u));
        B.row[at] = i;
        B.b[at] = e;
      }
      __syncwarp();
      bool any_out = false;
      for (int c0 = L.first(); c0 < n; c0 += 4 * L.step()) {
        float2 w[4];                     // four reads at a time
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = c0 + k * L.step();
          w[k] = L.live && c < n ? a.rec[(int64_t)B.b[c] * a.H + L.h] : make_float2(0.0f, 0.0f);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = c0 + k * L.step();
          if (c >= n) break;
          any_out |= marked(w[k].y);
          w2[c * a.hw + L.sub] = w[k];
        }
      }
      any_out = __any_sync(kFull, any_out);
      __syncwarp();
      for (int t0 = 0; t0 < n; t0 += U) {
        Vec<V> qq[U][SQ], gg[U][SV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = B.row[min(t0 + u, n - 1)];
          const char *q_row = row_at(a.q, r, a.ldq), *gy_row = row_at(a.gy, r, a.dv * 4u);
#pragma unroll
          for (int s = 0; s < SQ; ++s)
            qq[u][s] = s < SQ - 1 && !LOOSE ? load_vec<V, false>(q_row + oq[s], true)
                                            : load_vec<V, true>(q_row + oq[s], L.has(a.mq, s));
#pragma unroll
          for (int s = 0; s < SV; ++s)
            gg[u][s] = s < SV - 1 && !LOOSE ? load_vec<V, false>(gy_row + ov[s], true)
                                            : load_vec<V, true>(gy_row + ov[s], L.has(a.mv, s));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (t0 + u >= n) break;
          const float2 w = w2[(t0 + u) * a.hw + L.sub];
          if (any_out && marked(w.y)) continue;
#pragma unroll
          for (int s = 0; s < SQ; ++s)
#pragma unroll
            for (int c = 0; c < V; ++c) ak[s].x[c] = fmaf(w.x, qq[u][s].x[c], ak[s].x[c]);
#pragma unroll
          for (int s = 0; s < SV; ++s)
#pragma unroll
            for (int c = 0; c < V; ++c) av[s].x[c] = fmaf(w.y, gg[u][s].x[c], av[s].x[c]);
        }
      }
    }
    if constexpr (!WIDE) {
      if (t.W > 1) {
        const int warp = threadIdx.x >> 5;
        constexpr int T = (SQ + SV) * V;
        if (t.split > 0) {
#pragma unroll
          for (int s = 0; s < SQ; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) join[(warp * T + s * V + i) * 32 + lane] = ak[s].x[i];
#pragma unroll
          for (int s = 0; s < SV; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) join[(warp * T + (SQ + s) * V + i) * 32 + lane] = av[s].x[i];
        }
        __syncthreads();
        for (int o = 1; t.split == 0 && o < t.W; ++o) {
#pragma unroll
          for (int s = 0; s < SQ; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) ak[s].x[i] += join[((warp + o) * T + s * V + i) * 32 + lane];
#pragma unroll
          for (int s = 0; s < SV; ++s)
#pragma unroll
            for (int i = 0; i < V; ++i) av[s].x[i] += join[((warp + o) * T + (SQ + s) * V + i) * 32 + lane];
        }
      }
    }
    if (L.live && t.split == 0) {
#pragma unroll
      for (int s = 0; s < SQ; ++s) {
        if (!L.has(a.mq, s)) continue;
        if (t.part) {
          store_vec<V>(t.part + oq[s] / 4, ak[s]);
        } else if (a.gk) {
#pragma unroll
          for (int i = 0; i < V; ++i) ak[s].x[i] *= a.scale;
          store_vec<V>(a.gk + (int64_t)t.row * a.ldgk + oq[s] / 4, ak[s]);
        }
      }
#pragma unroll
      for (int s = 0; s < SV; ++s) {
        if (!L.has(a.mv, s)) continue;
        if (t.part) store_vec<V>(t.part + a.dq + ov[s] / 4, av[s]);
        else if (a.gv) store_vec<V>(a.gv + (int64_t)t.row * a.ldgv + ov[s] / 4, av[s]);
      }
    }
  }
}

// Joins the partial rows of the long rows, in window order: CTA w acts when such a row begins in window w,
// `cuts` CTAs a window share the row's floats, 128 at a time.  Its eight warps take every eighth window and
// are then added up in order.  Forward: the windows' sums meet at their common maximum.  Bound by the reads of the partials,
// one row for `win` edges' gathers of two.
constexpr int kJoinThreads = 256;

template <int PASS>   // 0: y, lse; 1: gq; 2: gk, gv
__device__ __forceinline__ void join_long_row(const AttnArgs& a, int cta, int cuts, const float* parts, int part_len) {
  __shared__ float top[32], total[32], sums[kJoinThreads / 32][128];
  const int32_t* ptr = PASS == 2 ? a.colptr : a.rowptr;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kJoinThreads / 32;
  const int cut = cta / a.n_win, w = cta - cut * a.n_win, first = w * a.win, end = min(first + a.win, a.E);
  int row, same;
  find_rows(ptr, a.N, end - 1, end - 1, row, same);   // the row pointers are the caller's: read before the wait
  wait_for_previous();
  if (row < 0) return;
  const int start = __ldg(ptr + row), stop = min(__ldg(ptr + row + 1), a.E);
  if (start < first || __ldg(ptr + row + 1) - start <= a.hub) return;
  const int n = (stop - 1) / a.win - w + 1;             // windows w .. w + n - 1; only the first may be slot 1
  auto part = [&](int i) {
    return parts + ((int64_t)(w + i) * 2 + (i == 0 && start > first ? 1 : 0)) * part_len;
  };
  if (PASS == 0) {
    for (int h = warp; h < a.H; h += warps) {
      float m = -INFINITY, l = 0.0f;
      for (int i = lane; i < n; i += 32) m = fmaxf(m, part(i)[part_len - 2 * a.H + h]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      const float ref = m == -INFINITY ? 0.0f : m;
      for (int i = lane; i < n; i += 32) {
        const float* p = part(i) + part_len - 2 * a.H + h;
        l += p[a.H] * exp_of(p[0] - ref);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
      if (lane == 0) {
        top[h] = ref;
        const bool none = m == -INFINITY && l == 0.0f;
        total[h] = none ? 0.0f : a.drop.inv_keep / l;
        if (a.lse && cut == 0) a.lse[(int64_t)row * a.H + h] = none ? -INFINITY : m + logf(l);
      }
    }
    __syncthreads();
  }
  const int width = PASS == 0 ? a.dv : PASS == 1 ? a.dq : a.dq + a.dv;
  for (int d0 = cut * 128; d0 < width; d0 += cuts * 128) {
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
        const float f = PASS == 0 ? exp_of(p[part_len - 2 * a.H + head[c]] - top[head[c]]) : 1.0f;
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

__global__ void __launch_bounds__(kJoinThreads) k_attn_fwd_join(const __grid_constant__ AttnArgs a) {
  join_long_row<0>(a, blockIdx.x, gridDim.x / a.n_win, a.part, a.part_len);
}

// What is left of a backward pass: the long rows of gq (CTAs 0 .. recv_joins - 1) and of gk and gv (the
// next send_joins), and the sums of gtable's partials.
struct Tail {
  int recv_joins, send_joins;
  float *recv_part, *send_part;
  int recv_len, send_len;
};

__global__ void __launch_bounds__(kJoinThreads) k_attn_bwd_tail(const __grid_constant__ AttnArgs a, const __grid_constant__ Tail t) {
  int cta = blockIdx.x;
  if (cta < t.recv_joins) return join_long_row<1>(a, cta, t.recv_joins / a.n_win, t.recv_part, t.recv_len);
  cta -= t.recv_joins;
  if (cta < t.send_joins) return join_long_row<2>(a, cta, t.send_joins / a.n_win, t.send_part, t.send_len);
  cta -= t.send_joins;
  wait_for_previous();
  table_sum(a, cta * (kJoinThreads / 32) + (threadIdx.x >> 5));
}

// Distance buckets: squares in 64 bits (products of 32-bit floats are exact there), a search by halving in
// shared memory, whose random reads are the limit.  A thread searches for its edges in step, so that the reads
// of one step overlap.  T = float: the squares rounded to 32 bits, which keeps their order, so the search can
// only go too far, and only past bounds that round to the distance's own value; the 64-bit squares then
// settle those.  3.0M edges: with 31 bounds 11.4 us in 64 bits and 13.9 in 32, with 255 bounds 28.9 and
// 18.0, with 63 15.7 and 13.3 (conflicts of the 8-byte reads grow with the bounds), hence T by the number of bounds.  Not kept:
// comparing with all of 32 bounds in turn, in 64 bits 16.5 us and in 32 bits 20.7 (instructions).
constexpr int kMaxBounds = 1023;
constexpr int kDoubleBounds = 31;

// PER edges a thread: four, whose 12 floats are three 16-byte reads, or one.
template <typename T, int PER>
__global__ void __launch_bounds__(256) k_buckets(int64_t E, const float* __restrict__ vec, int n, const float* __restrict__ bounds,
                                                 double cut2, int32_t* __restrict__ bucket) {
  __shared__ T b2[kMaxBounds + 1];       // padded with infinities to the next power of two
  __shared__ double exact[sizeof(T) == 8 ? 1 : kMaxBounds + 1];
  int half = n > 0 ? 1 : 0;              // the largest power of two in n
  while (2 * half <= n && half > 0) half *= 2;
  for (int i = threadIdx.x; i < 2 * half; i += 256) {
    double b = i < n ? (double)bounds[i] : INFINITY;
    b = b < 0.0 ? -1.0 : b * b;
    b2[i] = (T)b;
    if constexpr (sizeof(T) == 4) exact[i] = b;
  }
  __syncthreads();
  const int64_t thread = blockIdx.x * (int64_t)256 + threadIdx.x, threads = (int64_t)gridDim.x * 256;
  for (int64_t i = thread; i < (E + PER - 1) / PER; i += threads) {
    float v[3 * PER];
    const bool whole = PER == 1 || (i + 1) * PER <= E;
    if (PER == 4 && whole) {
      const float4* v4 = reinterpret_cast<const float4*>(vec) + 3 * i;
#pragma unroll
      for (int c = 0; c < 3 * PER / 4; ++c) {
        const float4 p = __ldg(v4 + c);
        v[4 * c] = p.x, v[4 * c + 1] = p.y, v[4 * c + 2] = p.z, v[4 * c + 3] = p.w;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 3 * PER; ++c) v[c] = 3 * PER * i + c < 3 * E ? __ldg(vec + 3 * PER * i + c) : 0.0f;
    }
    double d2[PER];
    T t2[PER];
    int k[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const double x = v[3 * e], y = v[3 * e + 1], z = v[3 * e + 2];
      d2[e] = x * x + y * y + z * z;
      t2[e] = (T)d2[e];
      k[e] = 0;
    }
    for (int step = half; step > 0; step >>= 1) {
#pragma unroll
      for (int e = 0; e < PER; ++e) k[e] += t2[e] >= b2[k[e] + step - 1] ? step : 0;
    }
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      k[e] = min(k[e], n);               // an infinite length passes the padding too
      if constexpr (sizeof(T) == 4) {
        while (k[e] > 0 && t2[e] == b2[k[e] - 1] && d2[e] < exact[k[e] - 1]) --k[e];
      }
      if (!(d2[e] < cut2)) k[e] = -1;
    }
    if (PER == 4 && whole) {
      reinterpret_cast<int4*>(bucket)[i] = make_int4(k[0], k[PER > 1 ? 1 : 0], k[PER > 2 ? 2 : 0], k[PER > 3 ? 3 : 0]);
    } else {
#pragma unroll
      for (int e = 0; e < PER; ++e)
        if (PER * i + e < E) bucket[PER * i + e] = k[e];
    }
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

// Launches `kernel` after the call's previous kernel (see let_next_launch).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = 1;
  count_launches(1);
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// Small tables (table_part): copies per CTA, one per group of lanes while they fit 512 bytes a thread (256 from 2^20
// edges on), 32 KB at most: behind the sender pass every CTA of that pass has this much shared memory too.  CTAs:
// enough that a group has no more than some 48 edges, while they stay eight a SM and a CTA has as many edges'
// values as it zeroes, sums and writes floats.  False where the latter leaves a group more than 128 edges, which
// is where k_attn_large_table takes over.  Whole backward pass in us with the one and the other, 8 heads: 46,080
// edges 64 buckets 42.5 / 49.3, 128 buckets 45.5 / 49.3, 192 58.6 / 51.2, 1,024 310 / 62; 3.0M edges 64 buckets
// 1,472 / 1,598, 96 1,829 / 1,602, 256 2,564 / 1,602.  512 against 256 bytes a thread: 165,448 edges, 82 buckets
// 733 / 741, 600,000 edges, 4 heads, 128 buckets 400 / 360, 3.0M edges, one head, 128 buckets 1,681 / 1,353.
bool small_table_plan(AttnArgs& a, int threads) {
  a.hist_lanes = 1;
  while (a.hist_lanes < a.H) a.hist_lanes *= 2;
  const int KH = std::max(1, a.K * a.H);
  const int floats = std::min(8 * 1024, (a.E < 1 << 20 ? 128 : 64) * threads);
  a.hist_copies = std::max(1, std::min(threads / a.hist_lanes, floats / KH));
  const int64_t want = std::max<int64_t>(1, (int64_t)a.E / std::max(a.hist_copies * 48, 4 * a.K));
  a.hist_ctas = (int)std::min<int64_t>(want, 148 * 2 * (kAttnThreads / std::min(threads, kAttnThreads)));
  return 4 * a.K <= 128 * a.hist_copies;
}

// Large ones (k_attn_large_table): CTAs of at least a tile of edges and as many edges as buckets, two a SM.
void large_table_plan(AttnArgs& a) {
  a.hist_lanes = 1;
  while (a.hist_lanes < a.H) a.hist_lanes *= 2;
  a.hist_copies = 1;
  a.hist_ctas = std::max(1, std::min(a.E / std::max(kTableTile, a.K), 148 * 2));
}

// Shared memory of a CTA of the one and of the other.
size_t small_table_bytes(const AttnArgs& a) { return sizeof(float) * (size_t)a.K * a.H * a.hist_copies; }
size_t large_table_bytes(const AttnArgs& a) { return sizeof(float) * ((size_t)a.K * a.H + kTableTile * (a.H + 1)); }

// Notes the threads of a pass's CTAs; a table behind the sender pass has CTAs of as many.
void plan_table(AttnArgs& a, int threads) {
  a.threads = threads;
  if (a.table_here) small_table_plan(a, threads);
}

template <int V, int SQ, int SV, bool LOOSE, bool WIDE>
cudaError_t launch_one(Pass pass, const AttnArgs& a, int threads, cudaStream_t s) {
  auto allow = [](auto kernel, size_t smem) {            // beyond 48 KB it has to be asked for
    return smem <= 48 * 1024 ? cudaSuccess : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  };
  size_t smem = batch_bytes(threads, a.hw);
  if (WIDE || a.W > 1) smem += sizeof(float) * join_floats(pass, V, SQ, SV, WIDE, rows_at_once(pass, V, SV, WIDE));
  const unsigned grid = (unsigned)(a.row_ctas + a.win_ctas);
  if (pass == kSend) {
    if (a.hist_ctas > 0) smem = std::max(smem, small_table_bytes(a));
    cudaError_t e = allow(k_attn_bwd_send<V, SQ, SV, LOOSE, WIDE>, smem);
    if (e != cudaSuccess) return e;
    return launch_after(k_attn_bwd_send<V, SQ, SV, LOOSE, WIDE>, grid + (unsigned)a.hist_ctas, threads, smem, s, a);
  }
  cudaError_t e = pass == kFwd ? allow(k_attn_fwd<V, SQ, SV, LOOSE, WIDE>, smem)
                               : allow(k_attn_bwd_recv<V, SQ, SV, LOOSE, WIDE>, smem);
  if (e != cudaSuccess) return e;
  if (pass == kFwd) k_attn_fwd<V, SQ, SV, LOOSE, WIDE><<<grid, threads, smem, s>>>(a);
  else k_attn_bwd_recv<V, SQ, SV, LOOSE, WIDE><<<grid, threads, smem, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

// The forms of the kernels for S chunks of v a lane: q with one or two chunks (logits from a few channels) or
// with S, where every lane has all but the last of each; and any others, where every read asks whether the
// lane has the chunk (100,003 edges with 28 floats a head of q and 63 of v, which fill two and four
// chunks: receiver pass 54 us in that form).
template <int V, int S>
cudaError_t launch_form(Pass pass, const AttnArgs& a, int cq, int cv, cudaStream_t s) {
  const int G = 32 / a.hw;
  auto fills = [G](int chunks, int slots) { return chunks >= (slots - 1) * G && chunks <= slots * G; };
  if (fills(cv, S)) {
    if (fills(cq, 1)) return launch_one<V, 1, S, false, false>(pass, a, a.W == 1 ? 32 : kAttnThreads, s);
    if constexpr (S > 2) {
      if (fills(cq, 2)) return launch_one<V, 2, S, false, false>(pass, a, a.W == 1 ? 32 : kAttnThreads, s);
    }
    if (fills(cq, S)) return launch_one<V, S, S, false, false>(pass, a, a.W == 1 ? 32 : kAttnThreads, s);
  }
  return launch_one<V, S, S, true, false>(pass, a, a.W == 1 ? 32 : kAttnThreads, s);
}

template <int V>
cudaError_t launch_slots(Pass pass, AttnArgs& a, cudaStream_t s) {
  const int cq = (a.mq.hd + V - 1) / V, cv = (a.mv.hd + V - 1) / V, chunks = std::max(cq, cv);
  if (chunks > 256) {
    int threads = 128;
    while (threads < kAttnWideThreads && (chunks + threads - 1) / threads > 4) threads *= 2;
    a.hw = 1;
    a.groups = a.H;
    a.W = 1;
    a.row_ctas = a.N * a.H;
    a.win_ctas = a.n_win;
    plan_table(a, threads);
    if (chunks <= 4 * threads) return launch_one<V, 4, 4, true, true>(pass, a, threads, s);
    return launch_one<V, 8, 8, true, true>(pass, a, threads, s);
  }
  // as many heads in a warp as leave a lane at most four chunks
  int hw = 1;
  while (hw < a.H && (chunks * 2 * hw + 31) / 32 <= 4) hw *= 2;
  a.hw = hw;
  a.groups = (a.H + hw - 1) / hw;
  const int need = (chunks + 32 / hw - 1) / (32 / hw);
  const int64_t units = (int64_t)a.N * a.groups;
  a.W = 1;
  while (a.W < kAttnWarps && units * a.W < 148 * 8 && a.E / std::max(1, a.N) >= 8 * a.W) a.W *= 2;
  const int per = a.W == 1 ? 1 : kAttnWarps / a.W;
  a.row_ctas = (int)((a.N + per - 1) / per) * a.groups;
  a.win_ctas = a.n_win * (a.W == 1 ? a.groups : 1);
  plan_table(a, a.W == 1 ? 32 : kAttnThreads);
  switch (need) {
    case 1: return launch_form<V, 1>(pass, a, cq, cv, s);
    case 2: return launch_form<V, 2>(pass, a, cq, cv, s);
    case 3: return launch_form<V, 3>(pass, a, cq, cv, s);
    case 4: return launch_form<V, 4>(pass, a, cq, cv, s);
    case 5:
    case 6: return launch_form<V, 6>(pass, a, cq, cv, s);
    default: return launch_form<V, 8>(pass, a, cq, cv, s);
  }
}

// Windows of 64 to 160 edges while there are four of them a SM, longer ones where there would be more than 16 a
// SM; rows of up to twice that stay with their own warps.  Fewer CTAs that look for long rows in vain against
// shorter ones for those there are.  With windows of 128 / 160 / 192 / 256 edges 162,892 edges without a long row
// take 213 / 210 / 208 / 208 us backward, 311,027 edges with a node of 8,192 neighbours 225 / 225 / 236 / 253;
// and with 160 edges against this rule 46,080 without a long row 16.5 against 17.0 us forward, 42,112 edges with
// a node of 2,942 neighbours 68 against 45, 10,834 edges in rows of up to 255 of 1,534 floats 129 against 72.
// Graphs of up to 320 edges do without the join's launch (192 edges: 4.7 us, 5.5 with it).
void window_plan(AttnArgs& a) {
  const auto each = [&](int per_sm) { return (a.E / (148 * per_sm) + 32) / 32 * 32; };
  a.win = std::max({kMinWindow, std::min(kFewWindows, each(4)), each(16)});
  a.hub = 2 * a.win;
  a.n_win = a.E > 2 * kFewWindows ? (a.E + a.win - 1) / a.win : 0;
}

// CTAs of the join of rows of `width` floats: as many a window as have 128 floats of the row each, while that
// keeps them to four a SM.  13,765 edges with a node of 1,617 neighbours, 672 floats a row: 75 us forward with one
// CTA a window, 68 so; with 16 a SM 66, but 46,080 edges without a long row 37.3 instead of 35.6 backward.
int join_ctas(const AttnArgs& a, int width) {
  return a.n_win * (a.n_win == 0 ? 0 : std::max(1, std::min((width + 127) / 128, 148 * 4 / a.n_win)));
}

int part_len(const AttnArgs& a, Pass pass) {
  const int n = pass == kFwd ? a.dv + 2 * a.H : pass == kRecv ? a.dq : a.dq + a.dv;
  return (n + 3) & ~3;
}

size_t part_bytes(const AttnArgs& a, Pass pass) { return sizeof(float) * 2 * (size_t)a.n_win * part_len(a, pass); }

// width: floats of a chunk.
cudaError_t launch_pass(Pass pass, AttnArgs& a, int width, float* part, cudaStream_t s) {
  a.part = part;
  a.part_len = part_len(a, pass);
  if (width == 4) return launch_slots<4>(pass, a, s);
  return width == 2 ? launch_slots<2>(pass, a, s) : launch_slots<1>(pass, a, s);
}

}  // namespace
}  // namespace tp

using namespace tp;

struct tp_attn_s {
  AttnArgs proto;
  int width;                 // the largest of 4, 2, 1 that divides every head's floats of every block
};

namespace {

struct BwdLayout {
  size_t rec, dst, hist, colptr, perm, scratch, recv_part, send_part, total;
};

BwdLayout bwd_layout(const tp_attn_s* h, int64_t N, int64_t E) {
  AttnArgs a = h->proto;
  a.N = (int)N;
  a.E = (int)E;
  window_plan(a);
  large_table_plan(a);
  int hist_ctas = a.hist_ctas;
  for (int threads : {32, kAttnThreads, 2 * kAttnThreads, kAttnWideThreads})       // whatever the passes will have
    if (small_table_plan(a, threads)) hist_ctas = std::max(hist_ctas, a.hist_ctas);
  BwdLayout L;
  size_t off = 0;
  const size_t e = (size_t)std::max<int64_t>(E, 1);
  L.rec = off;
  off += al256(sizeof(float2) * e * a.H);
  L.dst = off;
  off += al256(sizeof(int32_t) * e);
  L.hist = off;
  off += al256(sizeof(float) * (size_t)hist_ctas * a.K * a.H);
  L.colptr = off;
  off += al256(sizeof(int32_t) * (size_t)(N + 1));
  L.perm = off;
  off += al256(sizeof(int32_t) * e);
  L.scratch = off;
  off += al256(sizeof(int32_t) * (size_t)transpose_scratch_ints(N, E));
  L.recv_part = off;
  off += al256(part_bytes(a, kRecv));
  L.send_part = off;
  off += al256(part_bytes(a, kSend));
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
  if (ldq >= 1 << 30 || ldk >= 1 << 30 || ldv >= 1 << 30)
    return set_failure(TP_ERR_UNSUPPORTED, "row strides must stay below 2^30 floats");
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
  a.ldq = (uint32_t)(ldq * 4);
  a.ldk = (uint32_t)(ldk * 4);
  a.ldv = (uint32_t)(ldv * 4);
  a.table = table;
  a.scale = scale;
  window_plan(a);
  return TP_OK;
}

// The widest chunk, up to `width` floats, that pointers and row strides (in floats) allow.
int chunk_width(int width, std::initializer_list<const void*> pointers, std::initializer_list<int64_t> strides) {
  for (const void* p : pointers)
    while (reinterpret_cast<uintptr_t>(p) % (4 * width) != 0) width /= 2;
  for (int64_t ld : strides)
    while (ld % width != 0) width /= 2;
  return width;
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
  h.width = 4;
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
    for (int b = 0; b < side.map->nb; ++b)
      while (side.map->len[b] % h.width != 0) h.width /= 2;
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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int width = chunk_width(attn->width, {q, k, v, y}, {ldq, ldk, ldv});
  cudaError_t e = launch_pass(kFwd, a, width, static_cast<float*>(ws), s);
  if (e == cudaSuccess && a.n_win > 0) e = launch_after(k_attn_fwd_join, (unsigned)join_ctas(a, a.dv), kJoinThreads, 0, s, a);
  return cuda_status(e, "tp_attn_fwd");
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
  const int width = chunk_width(attn->width, {q, k, v, y, gy, gq, gk, gv},
                                {ldq, ldk, ldv, gq ? ldgq : 0, gk ? ldgk : 0, gv ? ldgv : 0});
  Tail tail{};
  tail.recv_part = reinterpret_cast<float*>(w + L.recv_part);
  tail.send_part = reinterpret_cast<float*>(w + L.send_part);
  tail.recv_len = part_len(a, kRecv);
  tail.send_len = part_len(a, kSend);
  tail.recv_joins = gq ? join_ctas(a, a.dq) : 0;
  tail.send_joins = send ? join_ctas(a, a.dq + a.dv) : 0;
  a.table_here = 0;
  a.hist_ctas = 0;
  e = launch_pass(kRecv, a, width, tail.recv_part, s);
  // a small table's CTAs come behind the sender pass's where there is one; its plan is the same without
  const bool table_wanted = gtable && E > 0, small = table_wanted && small_table_plan(a, a.threads);
  a.table_here = small && send;
  a.hist_ctas = 0;
  if (e == cudaSuccess && send) e = launch_pass(kSend, a, width, tail.send_part, s);
  if (e == cudaSuccess && table_wanted && !a.table_here) {
    // an ordinary launch: set up early, its few CTAs would gather on the SMs that the receiver pass leaves
    // first and run there one after another (162,892 edges: 46 instead of 16 us)
    if (small) {
      small_table_plan(a, a.threads);
      k_attn_table<<<a.hist_ctas, a.threads, small_table_bytes(a), s>>>(a);
    } else {
      large_table_plan(a);
      const size_t smem = large_table_bytes(a);
      if (smem > 48 * 1024) e = cudaFuncSetAttribute(k_attn_large_table, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e == cudaSuccess) k_attn_large_table<<<a.hist_ctas, kTableThreads, smem, s>>>(a);
    }
    if (e == cudaSuccess) {
      count_launches(1);
      e = cudaGetLastError();
    }
  }
  const int sums = a.hist_ctas > 1 ? (a.K * a.H + kJoinThreads / 32 - 1) / (kJoinThreads / 32) : 0;
  const unsigned rest = (unsigned)(tail.recv_joins + tail.send_joins + sums);
  if (e == cudaSuccess && rest > 0) e = launch_after(k_attn_bwd_tail, rest, kJoinThreads, 0, s, a, tail);
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
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const double cut2 = (double)cutoff * (double)cutoff;
  // four edges a thread only where that still fills the SMs
  const bool quad = al16(vec) && al16(bucket) && E >= 4 * 256 * 148;
  const int64_t per = quad ? 1024 : 256;
  const unsigned grid = (unsigned)std::min<int64_t>((E + per - 1) / per, 148 * 8);
  auto kernel = n_bounds <= kDoubleBounds ? (quad ? k_buckets<double, 4> : k_buckets<double, 1>)
                                          : (quad ? k_buckets<float, 4> : k_buckets<float, 1>);
  kernel<<<grid, 256, 0, s>>>(E, vec, n_bounds, bounds, cut2, bucket);
  count_launches(1);
  return cuda_status(cudaGetLastError(), "tp_distance_buckets");
}

}  // extern "C"
