// The counter-based generator of the dropout operators: Philox4x32-10 (Salmon, Moraes, Dror,
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  A block of four 32-bit words
// is a function of a 128-bit counter and a 64-bit key alone, so a mask is drawn again wherever
// it is needed and never stored.
#pragma once
#include <cmath>
#include <cstdint>

namespace tp {

struct DropArgs {
  const int64_t* rng;    // {seed, offset} in device memory; nullptr: no dropout
  int64_t site;          // added to the offset
  uint32_t threshold;    // a word below it drops its value
  float inv_keep;        // 1 / (1 - p)
};

struct DropKey {
  uint32_t k0, k1, c2, c3;
};

__device__ __forceinline__ DropKey drop_key(const DropArgs& d) {
  const uint64_t seed = (uint64_t)__ldg(reinterpret_cast<const long long*>(d.rng));
  const uint64_t off = (uint64_t)__ldg(reinterpret_cast<const long long*>(d.rng) + 1) + (uint64_t)d.site;
  return DropKey{(uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)off, (uint32_t)(off >> 32)};
}

__device__ __forceinline__ uint4 philox_block(const DropKey& key, uint64_t block) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = key.c2, c3 = key.c3;
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The four choices of a block, one byte each (1 = kept), value i of the block in byte i.
__device__ __forceinline__ uint32_t keep_bytes(const DropKey& key, uint32_t threshold, uint64_t block) {
  const uint4 w = philox_block(key, block);
  return (w.x >= threshold ? 1u : 0u) | (w.y >= threshold ? 0x100u : 0u) | (w.z >= threshold ? 0x10000u : 0u) |
         (w.w >= threshold ? 0x1000000u : 0u);
}

// False for p outside [0, 1) (NaN too), for one so near to 1 that every word would drop, and for
// p > 0 without rng.
inline bool drop_args(double p, const int64_t* rng, int64_t site, DropArgs& d) {
  d = DropArgs{nullptr, 0, 0u, 1.0f};
  if (!(p >= 0.0 && p < 1.0)) return false;
  if (p == 0.0) return true;
  const double t = std::nearbyint(p * 4294967296.0);
  if (!rng || t > 4294967295.0) return false;
  d = DropArgs{rng, site, (uint32_t)t, (float)(1.0 / (1.0 - p))};
  return true;
}

}  // namespace tp
