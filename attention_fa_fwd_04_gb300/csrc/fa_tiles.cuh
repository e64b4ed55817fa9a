// fa_tiles.cuh -- what the kernels that attend with 128-row tiles of query rows
// against 128-key tiles of a paged cache share (draft trees, shared prefixes):
// shapes, key masks, a tile's softmax, and their integer arithmetic.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "fa_ptx.cuh"

namespace fa {

namespace tiles {
constexpr int BM = 128;    // query rows per tile
constexpr int BN = 128;    // keys per K/V tile
constexpr int HALF_BYTES = 128 * 128;  // 128 rows x 64 elements x 2 bytes
constexpr int BAD_RING = 16;  // tiles whose page faults are remembered (> tiles in flight)
}  // namespace tiles

// a * b / c and a / c in 32 bits where they fit: a 64-bit division is a few
// hundred instructions, and a short call makes several one after another.
__device__ __forceinline__ long long mul_div(long long a, int b, long long c) {
  return a <= (0xffffffffll / (b + 1)) ? (long long)((uint32_t)a * (uint32_t)b / (uint32_t)c)
                                       : a * b / c;
}
__device__ __forceinline__ int div_small(long long a, int c) {
  return a >> 32 == 0 ? (int)((uint32_t)a / (uint32_t)c) : (int)(a / c);
}

// Bits [0, n) of a 128-bit mask held as two words (n may lie outside).
struct Mask128 {
  uint64_t lo, hi;
};
__device__ __forceinline__ uint64_t low_bits(int n) {
  return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1);
}
// Keys of a tile whose pages are sound (bad: one bit per box of `box` keys).
__device__ __forceinline__ Mask128 sound_keys(uint32_t bad, int box) {
  Mask128 m{~0ull, ~0ull};
  if (bad == 0) return m;
  for (int i = 0; i < 128 / box; ++i)
    if (bad >> i & 1) {
      const int a = i * box, e = a + box;
      m.lo &= ~(low_bits(e) & ~low_bits(a));
      m.hi &= ~(low_bits(e - 64) & ~low_bits(a - 64));
    }
  return m;
}

template <typename T>
struct TileType {
  static constexpr bool kBF16 = true;
  // Largest row sum of unnormalised P that a tile may leave before the row's
  // maximum is renewed: P fits the type and the sums fit fp32.
  static constexpr float kBig = 1.152921504606846976e18f;  // 2^60
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};
template <>
struct TileType<__half> {
  static constexpr bool kBF16 = false;
  static constexpr float kBig = 32768.f;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
};

// A row of Q (D elements; zeros if !real) as row `tid` of a 128-row tile, in the
// swizzled layout of a TMA load.
template <int D>
__device__ __forceinline__ void put_q_row(uint8_t* tile, int tid, const void* src, bool real) {
  uint4 v[D / 8];
#pragma unroll
  for (int x = 0; x < D / 8; ++x)
    v[x] = real ? static_cast<const uint4*>(src)[x] : make_uint4(0u, 0u, 0u, 0u);
  uint8_t* dst = tile + tid * 128;
#pragma unroll
  for (int x = 0; x < D / 8; ++x)
    *reinterpret_cast<uint4*>(dst + (x >> 3) * tiles::HALF_BYTES + (((x & 7) ^ (tid & 7)) << 4)) =
        v[x];
}

// Zeros into the rows of a V tile that are not in `keep`: warp wq of four takes 32
// of them, a row by D / 8 lanes.
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int wq, int lane, const Mask128& keep) {
  const uint64_t keep64 = wq < 2 ? keep.lo : keep.hi;
  const uint32_t clear = ~(uint32_t)(wq & 1 ? keep64 >> 32 : keep64);
  const int x = lane % (D / 8);
  uint8_t* const vt = tile + (x >> 3) * tiles::HALF_BYTES + wq * 32 * 128 + (x & 7) * 16;
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 256 / D) {
    const int r = r0 + lane / (D / 8);
    if (clear >> r & 1) *reinterpret_cast<uint4*>(vt + r * 128) = make_uint4(0u, 0u, 0u, 0u);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// Scores of the keys that are not in `see` become `hide`.
__device__ __forceinline__ void hide_keys(uint32_t (&sr)[4][32], const Mask128& see, float hide) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint64_t m64 = q < 2 ? see.lo : see.hi;
    const uint32_t m = (uint32_t)(q & 1 ? m64 >> 32 : m64);
    if (__all_sync(0xffffffffu, m == ~0u)) continue;
#pragma unroll
    for (int x = 0; x < 32; ++x)
      if (!(m >> x & 1)) sr[q][x] = __float_as_uint(hide);
  }
}

// One row's softmax over a tile: S from tensor memory at tS, P written back over
// it, the row's maximum *m_used (log2 units) and sum *l carried on.  c: scale *
// log2(e).  first: no tile came before.  mask(sr) hides scores (called if masked).
// settled(): waits until O at tO holds the tiles before; false gives up.
// A first tile takes its own maximum; later ones are exponentiated against the
// running one, and a warp takes the slow path only when a row's sum outgrows kBig or
// a row had seen no key yet.
// P is rounded to the inputs' type, which the matrix instructions take (half a step, 2^-8 or
// 2^-11, of sum p |v| / sum p); the sum is of P as it was, in fp32.
template <int D, typename T, typename Mask, typename Settled>
__device__ __forceinline__ bool softmax_tile(uint32_t tS, uint32_t tO, float c, bool first,
                                             bool masked, Mask&& mask, Settled&& settled,
                                             float* m_used, float* l) {
  constexpr float NEG_INF = -INFINITY;
  const bool neg = c < 0.f;
  uint32_t sr[4][32];
  float mx = neg ? -NEG_INF : NEG_INF;
  float2 la = make_float2(0.f, 0.f), lb = make_float2(0.f, 0.f);
  auto find_max = [&](uint32_t (&reg)[32]) {
    const float* v = reinterpret_cast<const float*>(reg);
    if (!neg) {
#pragma unroll
      for (int x = 0; x < 32; x += 2) mx = max3f(mx, v[x], v[x + 1]);
    } else {
#pragma unroll
      for (int x = 0; x < 32; x += 2) mx = min3f(mx, v[x], v[x + 1]);
    }
  };
  auto exp_store = [&](uint32_t (&reg)[32], int q, float top) {
    const float* v = reinterpret_cast<const float*>(reg);
    const float2 c2 = make_float2(c, c), nb = make_float2(-top, -top);
    uint32_t pk[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const float2 a = __ffma2_rn(make_float2(v[2 * t], v[2 * t + 1]), c2, nb);
      const float2 e = make_float2(fast_exp2(a.x), fast_exp2(a.y));
      if (t & 1)
        lb = __fadd2_rn(lb, e);
      else
        la = __fadd2_rn(la, e);
      pk[t] = TileType<T>::pack(e.x, e.y);
    }
    tmem_st16(tS + q * 16, pk);
  };
#pragma unroll
  for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, sr[q]);
  tmem_wait_ld();
#pragma unroll
  for (int q = 0; q < 4; ++q) reg_fence32(sr[q]);
  if (masked) mask(sr);
  bool renew = first;
  if (!renew) {
    const float top = *m_used == NEG_INF ? 0.f : *m_used;
#pragma unroll
    for (int q = 0; q < 4; ++q) exp_store(sr[q], q, top);
    const float lt = (la.x + la.y) + (lb.x + lb.y);
    const bool mine = !(lt <= TileType<T>::kBig) || *m_used == NEG_INF;
    renew = __any_sync(0xffffffffu, mine);
  }
  if (renew) {
#pragma unroll
    for (int q = 0; q < 4; ++q) find_max(sr[q]);
    const float m_new = fmaxf(*m_used, mx * c);
    const float f = *m_used == NEG_INF ? 0.f : fast_exp2(*m_used - m_new);
    const float top = m_new == NEG_INF ? 0.f : m_new;
    if (!first) {
      tmem_wait_st();
      la = lb = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) exp_store(sr[q], q, top);
    *l *= f;
    *m_used = m_new;
    if (!first) {
      if (!settled()) return false;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(tO + q * 32, o);
        tmem_wait_ld();
        reg_fence32(o);
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
        tmem_st32(tO + q * 32, o);
      }
    }
  }
  *l += (la.x + la.y) + (lb.x + lb.y);
  tmem_wait_st();
  return true;
}

}  // namespace fa
