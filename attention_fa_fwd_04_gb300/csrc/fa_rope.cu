// fa_rope.cu -- RMS norm of every query and key head and the rotation by
// position, in one pass: contiguous outputs, outputs straight into the pages
// of a KV cache, and the gradient.
//
// What it computes, for each head row x (D elements) of a token at position p:
//   y = x * r * w,  r = 1 / sqrt(mean(x^2) + eps),
//   and for each pair (a, b) of rotated elements, angle t = p * inv_freq[i]:
//   out_a = y_a cos t - y_b sin t,   out_b = y_b cos t + y_a sin t
//   (pairs (i, i + rot/2), or (2i, 2i + 1) when interleaved; elements at or
//   past rot pass through).
// Gradient, from g = dL/dout:
//   gy = g with every pair turned back by t,
//   dx = r (w gy) - x r^3 mean(x w gy),   dw = sum over rows of gy x r.
// Everything is held in fp32 and rounded once, to the outputs' type.
//
// HBM bound: one read and one write of the heads (gradient: two reads, one
// write), about ten fp32 operations per element.
//
// Layout: a head is D/16 lanes with two 16-byte chunks each, so that both
// elements of every pair sit in one lane (no exchange for the rotation; the
// mean takes log2(D/16) shuffles), and a warp holds 4 (D = 128) or 8 heads of
// one token.  A warp keeps one token's rotation in registers, as factors with
// the norm's weights in them, over all of that token's heads that it takes.
//
// Loads: a token's heads are contiguous, so each warp fetches steps of up to 16
// (D = 128) or 32 heads by one bulk copy into a ring of its own in shared
// memory, two steps ahead of its arithmetic: 128 to 192 KiB in flight per SM
// whatever the arithmetic's latency.  8192 tokens of 128 + 8 heads, D = 128: 98 us,
// 5.8 TB/s (84 us at the copy bandwidth); loads into registers, two head groups
// ahead, held 64 KiB in flight and took 117 us.
//
// Angles: positions reach 2^31, where an fp32 product p * inv_freq has no
// correct bit left.  Each block turns inv_freq once into a 64-bit fixed-point
// fraction of a turn; the phase p * fraction is then an integer product
// modulo 2^64 (whole turns drop out by overflow), good to about 2^-23 turns at
// |p| = 2^31 and to fp32 rounding below 2^28, without any 64-bit
// floating-point work per token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "fa.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

__device__ unsigned int g_rope_err = 0;

namespace rp {
constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int STAGE_BYTES = 4096;
// FEW: several tokens per step (see rope_few_kernel).
template <int D, bool BWD, bool FEW = false>
struct Cfg {
  static constexpr int STAGES = 3;  // steps in a warp's ring
  static constexpr int BLOCKS_PER_SM = 2;
  // Heads of a head group (one warp's registers): lanes hold two chunks of 8
  // elements of a head, in the gradient one.
  static constexpr int HPW = (BWD ? 256 : 512) / D;
  // A step fills a stage with heads (the gradient: with x and g of half as many).
  static constexpr int UNITS = 4;  // head groups per step
  static constexpr int HEADS = UNITS * HPW;
  // Tokens of a step, at most (FEW).
  static constexpr int TOKENS = FEW ? 384 / D : 1;
  // Rings, cosines and sines of a warp's tokens, turn fractions, barriers.
  static constexpr int TABLE = TOKENS * D;
  static constexpr int SMEM_CS = WARPS * TABLE * 4;
  static constexpr int SMEM_TOTAL =
      WARPS * STAGES * STAGE_BYTES + SMEM_CS + (D / 2) * 8 + WARPS * STAGES * 8 + 16;
};
}  // namespace rp

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
  return __half22float2(*reinterpret_cast<__half2*>(&u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Eight elements as four pairs for the packed fp32 operations.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float2 (&f)[4]) {
  f[0] = unpack2<T>(u.x);
  f[1] = unpack2<T>(u.y);
  f[2] = unpack2<T>(u.z);
  f[3] = unpack2<T>(u.w);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(pack2<T>(f[0].x, f[0].y), pack2<T>(f[1].x, f[1].y),
                    pack2<T>(f[2].x, f[2].y), pack2<T>(f[3].x, f[3].y));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 swap2(float2 v) { return make_float2(v.y, v.x); }

// One of the tensors a launch walks: queries, keys or values.
struct RopePart {
  const void* x;  // [tokens][H][D], token stride xs elements
  const void* g;  // gradient: dL/dout, contiguous
  void* y;        // contiguous output, or pages
  const void* w;  // [D]; null: copy the heads as they are (values)
  long long xs;
  int H;
  int paged;
  // Forward: the part's steps are [first, first + steps) of a token's.
  int first, steps;
  // Gradient, and few heads: blocks [b0, b0 + nb) of the grid walk the part, by
  // tasks of its own.
  int b0, nb;
  int spt, cpt;
  // Few heads: tokens per step; r * inv_h >> 16 = r / H for the rows of a step.
  int tg, inv_h;
};

struct RopeParams {
  RopePart part[3];
  int n_parts;
  const float* inv_freq;
  const int32_t* positions;  // [tokens]; null (paged only): the cache slot
  const int32_t* page_table;
  const int32_t* seqlens;
  int N;  // new tokens per sequence (paged)
  int page_size, max_pages, num_pages;
  int tokens;
  // A task is up to spt steps of one token, cpt tasks per token.
  int steps, spt, cpt;
  int rot;
  int inv_half;  // j * inv_half >> 16 = j / (rot / 2) for a step's table
  float eps;
  float* partial;  // gradient: [blocks][D] sums of dw
};

// Chunk positions and angle indexes of a lane (see the file's head).
template <int D, bool IL>
struct LaneMap {
  static constexpr int LPH = D / 16;  // lanes per head
  static constexpr int HPW = 32 / LPH;
  int sub, c0, c1;
  __device__ __forceinline__ LaneMap(int lane, int rot) {
    const int i = lane % LPH;
    sub = lane / LPH;
    if constexpr (IL) {
      c0 = i;
      c1 = i + LPH;
    } else {
      const int rc = rot / 16;
      c0 = i < rc ? i : 2 * rc + 2 * (i - rc);
      c1 = i < rc ? i + rc : c0 + 1;
    }
  }
  // Index of pair e's frequency, or -1 for elements that pass through.
  __device__ __forceinline__ int freq(int e, int rot) const {
    if constexpr (IL) {
      const int c = e < 4 ? c0 : c1;
      return c * 8 < rot ? c * 4 + (e & 3) : -1;
    } else {
      return c0 * 16 < rot ? c0 * 8 + e : -1;  // (c0 of other lanes is at least rot / 8)
    }
  }
};

__device__ __forceinline__ void load_fractions(const float* inv_freq, int n,
                                               unsigned long long* sF) {
  for (int i = threadIdx.x; i < n; i += rp::THREADS) {
    double t = (double)inv_freq[i] * 0.15915494309189533577;  // turns per position
    t -= floor(t);
    sF[i] = __double2ull_rn(t * 18446744073709551616.0);  // (t = 1 - 2^-53 still fits)
  }
  __syncthreads();
}

// Cosine and sine of a position's angle.  The phase's upper 32 bits are enough:
// 2^-32 turns are 2^-29 radians.  The nearest quarter turn is taken off exactly,
// and the Taylor series of what is left (at most pi / 4) end where their next
// term, r^11 / 11! and r^12 / 12!, is below 2^-28.  Within 1.7 * 2^-24 of the
// cosine and sine.  (sincospif reduces its argument itself: 32768 tokens of 8 + 2
// heads, D = 128, several tokens per step: 49.5 us with it, 48.4 so.)
__device__ __forceinline__ float2 cos_sin_at(unsigned long long fraction, int pos) {
  const uint32_t ph = (uint32_t)(fraction * (unsigned long long)(long long)pos >> 32);
  const uint32_t quarter = (ph + 0x20000000u) >> 30;
  const float r = (float)(int)(ph - (quarter << 30)) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float z = r * r;
  float s = fmaf(z, 1.f / 362880, -1.f / 5040), c = fmaf(z, -1.f / 3628800, 1.f / 40320);
  s = fmaf(z, s, 1.f / 120);
  c = fmaf(z, c, -1.f / 720);
  s = fmaf(z, s, -1.f / 6);
  c = fmaf(z, c, 1.f / 24);
  s = fmaf(z * s, r, r);
  c = fmaf(z, fmaf(z, c, -0.5f), 1.f);
  float2 v = quarter & 1 ? make_float2(s, c) : make_float2(c, s);
  if ((quarter + 1) & 2) v.x = -v.x;
  if (quarter & 2) v.y = -v.y;
  return v;
}
// Whole warp: cosines and then sines of a position's rot / 2 angles into the warp's
// table (each computed by one lane).
template <int D>
__device__ __forceinline__ void cos_sin(int rot, int pos, const unsigned long long* sF,
                                        float* table) {
  const int lane = threadIdx.x & 31;
  __syncwarp();  // (the table's last values have been read)
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const int f = lane + 32 * i;
    if (f < rot / 2) {
      const float2 v = cos_sin_at(sF[f], pos);
      table[f] = v.x;
      table[rot / 2 + f] = v.y;
    }
  }
  __syncwarp();
}
// The same for n tokens, lane l holding the l-th one's position: [token][rot].
__device__ __forceinline__ void cos_sin_group(const RopeParams& p, int n, int pos,
                                              const unsigned long long* sF, float* table) {
  const int lane = threadIdx.x & 31, half = p.rot / 2;
  __syncwarp();  // (the table's last values have been read)
#pragma unroll 2
  for (int j0 = 0; j0 < n * half; j0 += 32) {
    const int j = j0 + lane, t = j * p.inv_half >> 16;
    const int at = __shfl_sync(0xffffffffu, pos, t);
    if (j < n * half) {
      const float2 v = cos_sin_at(sF[j - t * half], at);
      table[t * half + j] = v.x;
      table[t * half + j + half] = v.y;
    }
  }
  __syncwarp();
}
// Four of a token's angles from the f-th on (f a multiple of 4), or 1 and 0 for
// elements that pass through (f < 0).
__device__ __forceinline__ void cos_sin_of(const float* table, int half, int f, float* cs,
                                           float* sn) {
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (f >= 0) {
    c = *reinterpret_cast<const float4*>(table + f);
    s = *reinterpret_cast<const float4*>(table + half + f);
  }
  cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
  sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
}

// The rotation as two products per output, o0 = x0 c0 + y0 s0 and o1 = x1 c1 +
// y1 s1, y the other element of each pair: for pairs across the chunks y0 = x1
// and y1 = x0, for neighbours the swapped x0 and x1.  The norm's weights go
// into the factors once per token.
template <bool IL>
struct Turn {
  float2 c0[4], s0[4], c1[4], s1[4];
  __device__ __forceinline__ void set(const float (&cs)[8], const float (&sn)[8],
                                      const float2 (&wa)[4], const float2 (&wb)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (IL) {
        c0[e] = make_float2(wa[e].x * cs[e], wa[e].y * cs[e]);
        s0[e] = make_float2(-wa[e].y * sn[e], wa[e].x * sn[e]);
        c1[e] = make_float2(wb[e].x * cs[e + 4], wb[e].y * cs[e + 4]);
        s1[e] = make_float2(-wb[e].y * sn[e + 4], wb[e].x * sn[e + 4]);
      } else {
        const float2 c = make_float2(cs[2 * e], cs[2 * e + 1]);
        const float2 n = make_float2(sn[2 * e], sn[2 * e + 1]);
        c0[e] = __fmul2_rn(wa[e], c);
        s0[e] = make_float2(-wb[e].x * n.x, -wb[e].y * n.y);
        c1[e] = __fmul2_rn(wb[e], c);
        s1[e] = __fmul2_rn(wa[e], n);
      }
    }
  }
  // a, b: the lane's chunks, turned and scaled by r.
  __device__ __forceinline__ void apply(float2 (&a)[4], float2 (&b)[4], float r) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 y0 = IL ? swap2(a[e]) : b[e], y1 = IL ? swap2(b[e]) : a[e];
      a[e] = __fmul2_rn(__ffma2_rn(a[e], c0[e], __fmul2_rn(y0, s0[e])), both(r));
      b[e] = __fmul2_rn(__ffma2_rn(b[e], c1[e], __fmul2_rn(y1, s1[e])), both(r));
    }
  }
};

// The gradient's lanes hold one chunk each, so its rotation (back, by the
// negative angle) is o = x c + y s with y the chunk that holds the pairs' other
// elements (neighbours: x swapped), read from the ring as well.  With half the
// registers per head, two head groups' chains run side by side within 128
// registers (16384 tokens of 16 + 16 heads, before later steps: 67.7 us; one after
// another at 80 registers and three blocks per SM 82 us; both chunks in a lane 89 us).
// Now 65.0 us, 6.2 TB/s.
template <int D, bool IL>
struct BackMap {
  static constexpr int LPH = D / 8;
  int sub, c, other;  // head of the group, chunk, the other elements' chunk
  float sign;
  int f0;  // first frequency, or -1
  __device__ __forceinline__ BackMap(int lane, int rot) {
    sub = lane / LPH;
    c = lane % LPH;
    other = c;
    sign = 1.f;
    f0 = -1;
    if (c * 8 >= rot) return;
    if constexpr (IL) {
      f0 = c * 4;
    } else {
      const int rc = rot / 16;
      const bool second = c >= rc;
      other = second ? c - rc : c + rc;
      sign = second ? -1.f : 1.f;
      f0 = (second ? other : c) * 8;
    }
  }
};
template <bool IL>
struct TurnBack {
  float2 c[4], s[4];
  __device__ __forceinline__ TurnBack() {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = both(1.f);
      s[e] = both(0.f);
    }
  }
  template <typename MAP>
  __device__ __forceinline__ void set(const float* table, int half, const MAP& m) {
    if (m.f0 < 0) return;  // (elements that pass through keep 1 and 0)
    const float4 c0 = *reinterpret_cast<const float4*>(table + m.f0);
    const float4 s0 = *reinterpret_cast<const float4*>(table + half + m.f0);
    if constexpr (IL) {
      c[0] = both(c0.x), c[1] = both(c0.y), c[2] = both(c0.z), c[3] = both(c0.w);
      s[0] = make_float2(s0.x, -s0.x);
      s[1] = make_float2(s0.y, -s0.y);
      s[2] = make_float2(s0.z, -s0.z);
      s[3] = make_float2(s0.w, -s0.w);
    } else {
      const float4 c1 = *reinterpret_cast<const float4*>(table + m.f0 + 4);
      const float4 s1 = *reinterpret_cast<const float4*>(table + half + m.f0 + 4);
      c[0] = make_float2(c0.x, c0.y);
      c[1] = make_float2(c0.z, c0.w);
      c[2] = make_float2(c1.x, c1.y);
      c[3] = make_float2(c1.z, c1.w);
      s[0] = __fmul2_rn(both(m.sign), make_float2(s0.x, s0.y));
      s[1] = __fmul2_rn(both(m.sign), make_float2(s0.z, s0.w));
      s[2] = __fmul2_rn(both(m.sign), make_float2(s1.x, s1.y));
      s[3] = __fmul2_rn(both(m.sign), make_float2(s1.z, s1.w));
    }
  }
};

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A warp's place in its tasks: warps take tasks in a grid stride, a step at a
// time.  (The stride is added as whole tokens and tasks: no division per task.)
struct RopeWalk {
  int t;        // token
  int c;        // task of the token
  int s;        // step of the token
  __device__ __forceinline__ RopeWalk(int w, int cpt, int spt) {
    t = w / cpt;
    c = w - t * cpt;
    s = c * spt;
  }
  __device__ __forceinline__ void next(int cpt, int spt, int steps, int dt, int dc) {
    ++s;
    if (s < steps && s < (c + 1) * spt) return;
    t += dt;
    c += dc;
    if (c >= cpt) {
      c -= cpt;
      ++t;
    }
    s = c * spt;
  }
};

// A lane's 16 bytes of a head in its ring.
__device__ __forceinline__ uint4 ring_load(const uint8_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// Shared memory of a block and of one of its warps.
template <int D, bool BWD, bool FEW = false>
struct RopeSmem {
  uint8_t* ring;
  float* table;
  unsigned long long* frac;
  uint64_t* full;
  volatile int* abort_flag;
  using C = rp::Cfg<D, BWD, FEW>;
  __device__ __forceinline__ RopeSmem(uint8_t* smem, int warp) {
    ring = smem + warp * C::STAGES * rp::STAGE_BYTES;
    uint8_t* q = smem + rp::WARPS * C::STAGES * rp::STAGE_BYTES;
    table = reinterpret_cast<float*>(q) + warp * C::TABLE;
    q += C::SMEM_CS;
    frac = reinterpret_cast<unsigned long long*>(q);
    q += (D / 2) * 8;
    full = reinterpret_cast<uint64_t*>(q) + warp * C::STAGES;
    q += rp::WARPS * C::STAGES * 8;
    abort_flag = reinterpret_cast<volatile int*>(q);
  }
};

// After an abort: the warp's loads in flight land before its block goes.
template <int STAGES>
__device__ __forceinline__ void drain_ring(uint64_t* full, uint32_t done, uint32_t issued) {
  for (uint32_t k = done; k < issued; ++k) mbar_wait_drain(&full[k % STAGES], (k / STAGES) & 1);
  __syncwarp();
}

// Cache row of token t (slot seqlens[b] - N + s), in rows of the pool, or -1
// (a padding sequence, or a length or page id out of range, which sets the
// bounds bit); *slot receives the position in the sequence.
__device__ __forceinline__ long long cache_row(const RopeParams& p, int t, int* slot) {
  const int b = t / p.N, s = t - b * p.N;
  const int L = p.seqlens[b];
  *slot = L - p.N + s;
  if (L < p.N) return -1;
  if (L > (long long)p.max_pages * p.page_size) {
    atomicOr(&g_rope_err, kErrBounds);
    return -1;
  }
  const int pg = *slot / p.page_size;
  const int pid = p.page_table[(size_t)b * p.max_pages + pg];
  if (pid < 0 || pid >= p.num_pages) {
    atomicOr(&g_rope_err, kErrBounds);
    return -1;
  }
  return (long long)pid * p.page_size + (*slot - pg * p.page_size);
}

// A token's steps are its query heads', then its keys', then (paged) its
// values'.
template <int D, typename T, bool IL, bool PAGED>
__global__ void __launch_bounds__(rp::THREADS, rp::Cfg<D, false>::BLOCKS_PER_SM)
    rope_kernel(const __grid_constant__ RopeParams p) {
  using C = rp::Cfg<D, false>;
  using M = LaneMap<D, IL>;
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RopeSmem<D, false> sm(smem, warp);
  if (lane == 0) {
    for (int i = 0; i < C::STAGES; ++i) mbar_init(&sm.full[i], 1);
    if (warp == 0) *sm.abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait_primary();
  const M m(lane, p.rot);
  const int warps = gridDim.x * rp::WARPS;
  const int dt = warps / p.cpt, dc = warps - dt * p.cpt;
  RopeWalk at(blockIdx.x * rp::WARPS + warp, p.cpt, p.spt), ahead = at;

  auto part_of = [&](int s) {
    int i = 0;
    if (p.n_parts > 1 && s >= p.part[1].first) i = 1;
    if (PAGED && p.n_parts > 2 && s >= p.part[2].first) i = 2;
    return i;
  };
  // The load of step `ahead` into its stage (k: the warp's step number).
  uint32_t issued = 0;
  auto fetch = [&]() {
    if (ahead.t >= p.tokens) return;
    if (lane == 0) {
      const RopePart& pt = p.part[part_of(ahead.s)];
      const int h0 = (ahead.s - pt.first) * C::HEADS;
      const uint32_t bytes = (uint32_t)(pt.H - h0 < C::HEADS ? pt.H - h0 : C::HEADS) * D * 2;
      const int st = issued % C::STAGES;
      mbar_arrive_expect_tx(&sm.full[st], bytes);
      bulk_load(sm.ring + st * rp::STAGE_BYTES,
                static_cast<const T*>(pt.x) + ahead.t * pt.xs + (size_t)h0 * D, bytes,
                &sm.full[st]);
    }
    ++issued;
    ahead.next(p.cpt, p.spt, p.steps, dt, dc);
  };
  __syncwarp();
  for (int i = 0; i < C::STAGES; ++i) fetch();
  int pos_n = 0;
  if ((!PAGED || p.positions) && at.t < p.tokens) pos_n = p.positions[at.t];
  load_fractions(p.inv_freq, p.rot / 2, sm.frac);  // (ends with the block's barrier)

  int token = -1;
  long long row = 0;
  int kind = -1;  // the part that `turn` holds the weights of
  float cs[8], sn[8];
  Turn<IL> turn;
  uint32_t k = 0;
  for (; at.t < p.tokens; ++k) {
    const int pos = pos_n;
    RopeWalk nx = at;
    nx.next(p.cpt, p.spt, p.steps, dt, dc);
    if ((!PAGED || p.positions) && nx.t < p.tokens) pos_n = p.positions[nx.t];
    const int i = part_of(at.s);
    const RopePart& pt = p.part[i];
    if (at.t != token) {  // warp-uniform, as is every branch on the walk
      token = at.t;
      kind = -1;
      int slot = 0;
      if constexpr (PAGED) row = cache_row(p, token, &slot);
      if (pt.w) {
        cos_sin<D>(p.rot, PAGED && !p.positions ? slot : pos, sm.frac, sm.table);
        cos_sin_of(sm.table, p.rot / 2, m.freq(0, p.rot), cs, sn);
        cos_sin_of(sm.table, p.rot / 2, m.freq(4, p.rot), cs + 4, sn + 4);
      }
    }
    float2 a[4], b[4];
    if (i != kind) {
      kind = i;
      if (!PAGED || pt.w) {
        unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(pt.w) + m.c0 * 8), a);
        unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(pt.w) + m.c1 * 8), b);
        turn.set(cs, sn, a, b);
      }
    }
    const int h0 = (at.s - pt.first) * C::HEADS;
    const int nh = pt.H - h0 < C::HEADS ? pt.H - h0 : C::HEADS;
    const long long to = PAGED && pt.paged ? row : token;
    T* y = static_cast<T*>(pt.y) + (to * pt.H + h0 + m.sub) * D;
    const uint8_t* x = sm.ring + (k % C::STAGES) * rp::STAGE_BYTES + m.sub * D * 2;
    if (!mbar_wait<true>(&sm.full[k % C::STAGES], (k / C::STAGES) & 1, sm.abort_flag,
                         &g_rope_err, 20))
      break;
    __syncwarp();
#pragma unroll
    for (int u = 0; u < C::UNITS; ++u) {
      if (u * C::HPW >= nh) break;  // warp-uniform
      uint4 r0 = ring_load(x + u * C::HPW * D * 2 + m.c0 * 16);
      uint4 r1 = ring_load(x + u * C::HPW * D * 2 + m.c1 * 16);
      if (!PAGED || pt.w) {
        unpack8<T>(r0, a);
        unpack8<T>(r1, b);
        float2 s2 = both(0.f), t2 = both(0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s2 = __ffma2_rn(a[e], a[e], s2);
          t2 = __ffma2_rn(b[e], b[e], t2);
        }
        const float ss = head_sum<M::LPH>((s2.x + s2.y) + (t2.x + t2.y));
        turn.apply(a, b, rsqrtf(ss * (1.f / D) + p.eps));
        r0 = pack8<T>(a);
        r1 = pack8<T>(b);
      }
      if (u * C::HPW + m.sub < nh && (!PAGED || to >= 0)) {
        *reinterpret_cast<uint4*>(y + u * C::HPW * D + m.c0 * 8) = r0;
        *reinterpret_cast<uint4*>(y + u * C::HPW * D + m.c1 * 8) = r1;
      }
    }
    __syncwarp();  // the stage has been read
    fetch();
    at = nx;
  }
  if (*sm.abort_flag) drain_ring<C::STAGES>(sm.full, k, issued);
}

// Few heads per token: a step takes several tokens, so that it still fills the
// lanes and moves a few KB.  Blocks walk one part each, as in the gradient; a
// step's rows are its tokens' heads one after another, the table holds the
// cosines and sines of its tokens, and each lane makes the factors of its own
// row's token.  50640 tokens of 4 + 2 heads, D = 64: 19.9 us, 3.9 TB/s (11.5 us at
// the copy bandwidth); bound by latency: 16 warps per SM, each on one chain of
// shuffles, a reciprocal root and its factors, leave half of the issue slots free.
// With one head a step is 384 / D rows, a quarter of a head group at D = 64: 60000
// tokens of 1 + 1 heads 18.6 us against 4.5.

// Copies of a step's heads of the tokens [t0, t0 + n) into `to`; whole warp.
template <int D, typename T>
__device__ __forceinline__ void fetch_group(const void* x, long long xs, int H, long long t0, int n,
                                            uint8_t* to, uint64_t* bar) {
  const int lane = threadIdx.x & 31;
  const uint32_t bytes = (uint32_t)H * D * 2;
  const T* src = static_cast<const T*>(x) + t0 * xs;
  if (xs == (long long)H * D) {
    if (lane == 0) bulk_load(to, src, n * bytes, bar);
  } else if (lane < n) {
    bulk_load(to + lane * bytes, src + lane * xs, bytes, bar);
  }
}

template <int D, typename T, bool IL, bool PAGED>
__global__ void __launch_bounds__(rp::THREADS, rp::Cfg<D, false, true>::BLOCKS_PER_SM)
    rope_few_kernel(const __grid_constant__ RopeParams p) {
  using C = rp::Cfg<D, false, true>;
  using M = LaneMap<D, IL>;
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RopeSmem<D, false, true> sm(smem, warp);
  if (lane == 0) {
    for (int i = 0; i < C::STAGES; ++i) mbar_init(&sm.full[i], 1);
    if (warp == 0) *sm.abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait_primary();
  const M m(lane, p.rot);
  int part = 0;
  if (p.n_parts > 1 && (int)blockIdx.x >= p.part[1].b0) part = 1;
  if (PAGED && p.n_parts > 2 && (int)blockIdx.x >= p.part[2].b0) part = 2;
  const RopePart& pt = p.part[part];
  const int H = pt.H, tg = pt.tg, half = p.rot / 2;
  const int groups = (p.tokens + tg - 1) / tg, warps = pt.nb * rp::WARPS;
  int at = (blockIdx.x - pt.b0) * rp::WARPS + warp, ahead = at;
  uint32_t issued = 0;
  auto tokens_of = [&](int g) { return p.tokens - g * tg < tg ? p.tokens - g * tg : tg; };
  auto fetch = [&]() {
    if (ahead >= groups) return;
    const int n = tokens_of(ahead), st = issued % C::STAGES;
    if (lane == 0) mbar_arrive_expect_tx(&sm.full[st], (uint32_t)n * H * D * 2);
    __syncwarp();
    fetch_group<D, T>(pt.x, pt.xs, H, (long long)ahead * tg, n, sm.ring + st * rp::STAGE_BYTES,
                      &sm.full[st]);
    ++issued;
    ahead += warps;
  };
  __syncwarp();
  for (int i = 0; i < C::STAGES; ++i) fetch();
  const bool own_pos = !PAGED || p.positions, normed = !PAGED || pt.w;
  auto position = [&](int g) {
    return own_pos && normed && g < groups && lane < tokens_of(g) ? p.positions[g * tg + lane] : 0;
  };
  int pos_n = position(at);
  float2 wa[4], wb[4];
  if (normed) {
    unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(pt.w) + m.c0 * 8), wa);
    unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(pt.w) + m.c1 * 8), wb);
  }
  load_fractions(p.inv_freq, half, sm.frac);  // (ends with the block's barrier)

  uint32_t k = 0;
  for (; at < groups; at += warps, ++k) {
    const int n = tokens_of(at), rows = n * H;
    int pos = pos_n;
    pos_n = position(at + warps);
    long long row = 0;
    if constexpr (PAGED) {
      if (lane < n && (pt.paged || !own_pos)) {
        int slot;
        row = cache_row(p, at * tg + lane, &slot);
        if (!own_pos) pos = slot;
      }
    }
    if (normed) cos_sin_group(p, n, pos, sm.frac, sm.table);
    T* const y = static_cast<T*>(pt.y) + (long long)at * tg * H * D;
    const uint8_t* x = sm.ring + (k % C::STAGES) * rp::STAGE_BYTES + m.sub * D * 2;
    if (!mbar_wait<true>(&sm.full[k % C::STAGES], (k / C::STAGES) & 1, sm.abort_flag,
                         &g_rope_err, 20))
      break;
    __syncwarp();
    Turn<IL> turn;
    int turned = -1;  // the token whose factors `turn` holds
    for (int u = 0; u * C::HPW < rows; ++u) {
      // (A lane past the last row works on what its ring holds.)
      const int r = u * C::HPW + m.sub;
      int t = r * pt.inv_h >> 16;
      t = t < n ? t : n - 1;
      uint4 r0 = ring_load(x + u * C::HPW * D * 2 + m.c0 * 16);
      uint4 r1 = ring_load(x + u * C::HPW * D * 2 + m.c1 * 16);
      if (normed) {
        float2 a[4], b[4];
        unpack8<T>(r0, a);
        unpack8<T>(r1, b);
        float2 s2 = both(0.f), t2 = both(0.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s2 = __ffma2_rn(a[e], a[e], s2);
          t2 = __ffma2_rn(b[e], b[e], t2);
        }
        if (t != turned) {
          turned = t;
          float cs[8], sn[8];
          cos_sin_of(sm.table + t * p.rot, half, m.freq(0, p.rot), cs, sn);
          cos_sin_of(sm.table + t * p.rot, half, m.freq(4, p.rot), cs + 4, sn + 4);
          turn.set(cs, sn, wa, wb);
        }
        const float ss = head_sum<M::LPH>((s2.x + s2.y) + (t2.x + t2.y));
        turn.apply(a, b, rsqrtf(ss * (1.f / D) + p.eps));
        r0 = pack8<T>(a);
        r1 = pack8<T>(b);
      }
      T* dst = y + r * D;
      bool real = r < rows;
      if constexpr (PAGED) {
        const long long to = __shfl_sync(0xffffffffu, row, t);
        if (pt.paged) {
          dst = static_cast<T*>(pt.y) + (to * H + (r - t * H)) * D;
          real = real && to >= 0;
        }
      }
      if (real) {
        *reinterpret_cast<uint4*>(dst + m.c0 * 8) = r0;
        *reinterpret_cast<uint4*>(dst + m.c1 * 8) = r1;
      }
    }
    __syncwarp();  // the stage has been read
    fetch();
  }
  if (*sm.abort_flag) drain_ring<C::STAGES>(sm.full, k, issued);
}

// Gradient of rope_kernel.  Each block walks the queries or the keys, and ends
// with one row of partial[] (its sum of gy x r per column); the sums of a
// lane, a block and the blocks are taken in a fixed order, so equal calls give
// equal bits.
// FEW: steps of several tokens, as in rope_few_kernel (walked as groups of one
// step each).
template <int D, typename T, bool IL, bool FEW>
__global__ void __launch_bounds__(rp::THREADS, rp::Cfg<D, true, FEW>::BLOCKS_PER_SM)
    rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  using C = rp::Cfg<D, true, FEW>;
  using M = BackMap<D, IL>;
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RopeSmem<D, true, FEW> sm(smem, warp);
  if (lane == 0) {
    for (int i = 0; i < C::STAGES; ++i) mbar_init(&sm.full[i], 1);
    if (warp == 0) *sm.abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait_primary();
  const M m(lane, p.rot);
  const RopePart& pt = p.part[p.n_parts > 1 && (int)blockIdx.x >= p.part[1].b0 ? 1 : 0];
  const int warps = pt.nb * rp::WARPS;
  const int dt = warps / pt.cpt, dc = warps - dt * pt.cpt;
  const int tg = FEW ? pt.tg : 1, items = FEW ? (p.tokens + tg - 1) / tg : p.tokens;
  auto tokens_of = [&](int g) { return p.tokens - g * tg < tg ? p.tokens - g * tg : tg; };
  RopeWalk at((blockIdx.x - pt.b0) * rp::WARPS + warp, pt.cpt, pt.spt), ahead = at;
  uint32_t issued = 0;
  // x in the first half of the stage, g in the second.
  auto fetch = [&]() {
    if (ahead.t >= items) return;
    if constexpr (FEW) {
      const int n = tokens_of(ahead.t), st = issued % C::STAGES;
      const long long t0 = (long long)ahead.t * tg;
      uint8_t* to = sm.ring + st * rp::STAGE_BYTES;
      if (lane == 0) mbar_arrive_expect_tx(&sm.full[st], (uint32_t)n * pt.H * D * 4);
      __syncwarp();
      fetch_group<D, T>(pt.x, pt.xs, pt.H, t0, n, to, &sm.full[st]);
      fetch_group<D, T>(pt.g, (long long)pt.H * D, pt.H, t0, n, to + rp::STAGE_BYTES / 2,
                        &sm.full[st]);
    } else if (lane == 0) {
      const int h0 = ahead.s * C::HEADS;
      const uint32_t bytes = (uint32_t)(pt.H - h0 < C::HEADS ? pt.H - h0 : C::HEADS) * D * 2;
      const int st = issued % C::STAGES;
      uint8_t* to = sm.ring + st * rp::STAGE_BYTES;
      mbar_arrive_expect_tx(&sm.full[st], 2 * bytes);
      bulk_load(to, static_cast<const T*>(pt.x) + ahead.t * pt.xs + (size_t)h0 * D, bytes,
                &sm.full[st]);
      bulk_load(to + rp::STAGE_BYTES / 2,
                static_cast<const T*>(pt.g) + ((long long)ahead.t * pt.H + h0) * D, bytes,
                &sm.full[st]);
    }
    ++issued;
    ahead.next(pt.cpt, pt.spt, pt.steps, dt, dc);
  };
  __syncwarp();
  for (int i = 0; i < C::STAGES; ++i) fetch();
  // FEW: lane l holds the l-th token's.
  auto position = [&](int g) {
    if constexpr (FEW) return g < items && lane < tokens_of(g) ? p.positions[g * tg + lane] : 0;
    return g < items ? p.positions[g] : 0;
  };
  int pos_n = position(at.t);
  float2 w[4];
  unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(pt.w) + m.c * 8), w);
  load_fractions(p.inv_freq, p.rot / 2, sm.frac);
  float2 acc[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = both(0.f);
  int token = -1;
  TurnBack<IL> back;
  uint32_t k = 0;
  for (; at.t < items; ++k) {
    const int pos = pos_n;
    RopeWalk nx = at;
    nx.next(pt.cpt, pt.spt, pt.steps, dt, dc);
    if (FEW || nx.t < items) pos_n = position(nx.t);
    int h0 = 0, nh;  // first head and number of rows
    if constexpr (FEW) {
      token = at.t * tg;
      nh = tokens_of(at.t) * pt.H;
      cos_sin_group(p, tokens_of(at.t), pos, sm.frac, sm.table);
    } else {
      if (at.t != token) {
        token = at.t;
        cos_sin<D>(p.rot, pos, sm.frac, sm.table);
        back.set(sm.table, p.rot / 2, m);
      }
      h0 = at.s * C::HEADS;
      nh = pt.H - h0 < C::HEADS ? pt.H - h0 : C::HEADS;
    }
    T* dst = static_cast<T*>(pt.y) + ((long long)token * pt.H + h0 + m.sub) * D;
    const uint8_t* x = sm.ring + (k % C::STAGES) * rp::STAGE_BYTES + m.sub * D * 2;
    if (!mbar_wait<true>(&sm.full[k % C::STAGES], (k / C::STAGES) & 1, sm.abort_flag,
                         &g_rope_err, 21))
      break;
    __syncwarp();
    auto unit = [&](int u) {
      // (A lane past the last head works on what its ring holds, and its
      // terms are left out of the weights' sums.)
      const bool real = u * C::HPW + m.sub < nh;
      TurnBack<IL> own;
      if constexpr (FEW) {
        int t = (u * C::HPW + m.sub) * pt.inv_h >> 16;
        t = t < C::TOKENS ? t : 0;  // (of a lane past the last head: any)
        own.set(sm.table + t * p.rot, p.rot / 2, m);
      }
      const TurnBack<IL>& by = FEW ? own : back;
      const uint8_t* xu = x + u * C::HPW * D * 2;
      const uint8_t* gu = xu + rp::STAGE_BYTES / 2;
      float2 a[4], g[4], y[4];
      unpack8<T>(ring_load(xu + m.c * 16), a);
      unpack8<T>(ring_load(gu + m.c * 16), g);
      if constexpr (!IL) unpack8<T>(ring_load(gu + m.other * 16), y);
      float2 s2 = both(0.f), d2 = both(0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] = __ffma2_rn(g[e], by.c[e], __fmul2_rn(IL ? swap2(g[e]) : y[e], by.s[e]));
        y[e] = __fmul2_rn(g[e], a[e]);
        s2 = __ffma2_rn(a[e], a[e], s2);
        d2 = __ffma2_rn(y[e], w[e], d2);
      }
      float ss = s2.x + s2.y, dot = d2.x + d2.y;
#pragma unroll
      for (int o = M::LPH / 2; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
      const float nf = -dot * (1.f / D) * r * r;  // -r^2 mean(x w gy)
      if (real) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[e] = __ffma2_rn(y[e], both(r), acc[e]);
          a[e] = __fmul2_rn(__ffma2_rn(a[e], both(nf), __fmul2_rn(w[e], g[e])), both(r));
        }
        *reinterpret_cast<uint4*>(dst + u * C::HPW * D + m.c * 8) = pack8<T>(a);
      }
    };
    if (nh == C::HEADS) {
#pragma unroll 2
      for (int u = 0; u < C::UNITS; ++u) unit(u);
    } else {
#pragma unroll 1
      for (int u = 0; u * C::HPW < nh; ++u) unit(u);
    }
    __syncwarp();  // the stage has been read
    fetch();
    at = nx;
  }
  if (*sm.abort_flag) drain_ring<C::STAGES>(sm.full, k, issued);
  __syncthreads();  // the rings have been read: they take the block's sums
  float* sW = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float v = e & 1 ? acc[e >> 1].y : acc[e >> 1].x;
#pragma unroll
    for (int o = M::LPH; o < 32; o <<= 1)  // the lanes of the warp's other heads
      v += __shfl_xor_sync(0xffffffffu, v, o);
    if (m.sub == 0) sW[warp * D + m.c * 8 + e] = v;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < rp::WARPS; ++i) s += sW[i * D + threadIdx.x];
    p.partial[(size_t)blockIdx.x * D + threadIdx.x] = s;
  }
}

// dw of part blockIdx.y: the sum of its blocks' partial rows, 32 columns per
// block; each of the 32 warps sums every 32nd row, then one column.
constexpr int kDwThreads = 1024;
__global__ void __launch_bounds__(kDwThreads)
    rope_dw_kernel(const float* partial, int D, int b0q, int nbq, float* dqw, int b0k, int nbk,
                   float* dkw) {
  __shared__ float sS[32][33];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int b0 = blockIdx.y ? b0k : b0q, nb = blockIdx.y ? nbk : nbq;
  float* dw = blockIdx.y ? dkw : dqw;
  if (!dw) return;
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  const float* col = partial + (size_t)b0 * D + blockIdx.x * 32 + lane;
  float s = 0.f;
#pragma unroll 8
  for (int i = r; i < nb; i += 32) s += col[(size_t)i * D];
  sS[r][lane] = s;
  __syncthreads();
  s = sS[lane][r];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) dw[blockIdx.x * 32 + r] = s;
}

// Steps per task: the fewest rounds of the resident warps, a round costing its
// steps and, once, the token's cosines, sines and factors.  These count as an
// eighth of a step (forward: 8192 tokens of 32 + 8 heads 30.5 us so, 31.5 us as a
// quarter; 8192 of 128 + 8 heads 97.9 us, 100.9 us as a sixteenth) or a sixteenth
// (gradient: 16384 tokens of 16 + 16 heads 65.0 us so, 69.0 us as an eighth).
static void plan_tasks(int tokens, int steps, long long warps, int weight, int* spt, int* cpt) {
  long long best = 0;
  for (int c = 1; c <= steps && c <= 64; ++c) {
    const int u = (steps + c - 1) / c;
    if ((steps + u - 1) / u != c) continue;
    const long long cost = ((long long)tokens * c + warps - 1) / warps * (weight * u + 1);
    if (best == 0 || cost < best) {
      best = cost;
      *spt = u;
      *cpt = c;
    }
  }
}

// Blocks of the parts, in proportion to what a token of each costs, all of them
// resident at once (left: what the parts before this one did not take).
static int part_blocks(const RopeParams& p, int i, long long slots, const long long* cost,
                       long long left) {
  long long all = 0;
  for (int k = 0; k < p.n_parts; ++k) all += cost[k];
  long long nb = i + 1 < p.n_parts ? (slots * cost[i] + all / 2) / all : left;
  if (nb > left - (p.n_parts - 1 - i)) nb = left - (p.n_parts - 1 - i);
  return (int)(nb < 1 ? 1 : nb);
}

// Steps of several tokens, where each part's step has room for a second token and
// there are tokens enough for more than one.  A part's step holds as many tokens
// as take the fewest rounds of its warps, a round costing its head groups and
// about two more.  Returns the grid size, or 0.
// (D = 64, 50640 tokens of 4 + 2 heads: 19.9 us, a token per step 50.5; 16384 of
// 16 + 16: 24.8 and 28.5; without room, 16384 of 32 + 4: 32.7 and 31.8, and D = 128,
// 16384 of 16 + 4: 35.5 and 32.2.  Into pages, 4096 of 8 + 2 + 2: D = 64 7.0 and
// 9.5, D = 128 11.7 and 10.9.  Gradient: 33841 of 8 + 4 heads 35.0 and 40.9;
// without room, D = 128, 32768 of 8 + 2: 73.3 and 60.4.)
static int plan_few(RopeParams* p, int D, bool bwd, long long slots) {
  const int heads = (bwd ? rp::Cfg<128, true>::HEADS : rp::Cfg<128, false>::HEADS) * 128 / D;
  const int hpw = heads / rp::Cfg<128, false>::UNITS, most = 384 / D;
  long long cost[3] = {0, 0, 0};
  for (int i = 0; i < p->n_parts; ++i) {
    const int H = p->part[i].H;
    if (2 * H > heads) return 0;
    const int tg = heads / H < most ? heads / H : most;
    const int unit = p->part[i].w ? 5 : 2;  // (values are only copied)
    cost[i] = 1024ll * (unit * ((tg * H + hpw - 1) / hpw) + 10) / tg;
  }
  long long left = slots;
  int b0 = 0;
  bool several = false;
  for (int i = 0; i < p->n_parts; ++i) {
    RopePart& t = p->part[i];
    long long nb = part_blocks(*p, i, slots, cost, left);
    left -= nb;
    long long best = 0;
    for (int tg = 1; tg <= most && tg * t.H <= heads; ++tg) {
      const long long groups = ((long long)p->tokens + tg - 1) / tg, warps = nb * rp::WARPS;
      const long long c = (groups + warps - 1) / warps * ((tg * t.H + hpw - 1) / hpw + 2);
      if (best == 0 || c < best) {
        best = c;
        t.tg = tg;
      }
    }
    several |= t.tg > 1;
    const long long need =
        (((long long)p->tokens + t.tg - 1) / t.tg + rp::WARPS - 1) / rp::WARPS;
    if (nb > need) nb = need;
    t.inv_h = 65536 / t.H + 1;
    t.steps = t.spt = t.cpt = 1;
    t.b0 = b0;
    t.nb = (int)nb;
    b0 += t.nb;
  }
  p->inv_half = 65536 / (p->rot / 2) + 1;
  return several ? b0 : 0;
}

// Steps, tasks and blocks.  Returns the grid size.
static int plan_parts(RopeParams* p, int D, bool bwd, bool* few) {
  const int heads = (bwd ? rp::Cfg<128, true>::HEADS : rp::Cfg<128, false>::HEADS) * 128 / D;
  const int hpw = heads / rp::Cfg<128, false>::UNITS;
  const int sms = sm_count() > 0 ? sm_count() : 148;
  const long long slots =  // resident blocks
      (long long)sms *
      (bwd ? rp::Cfg<128, true>::BLOCKS_PER_SM : rp::Cfg<128, false>::BLOCKS_PER_SM);
  const int blocks = plan_few(p, D, bwd, slots);
  *few = blocks > 0;
  if (*few) return blocks;
  long long steps = 0, cost[3];
  for (int i = 0; i < p->n_parts; ++i) {
    RopePart& t = p->part[i];
    t.steps = (t.H + heads - 1) / heads;
    t.first = (int)steps;
    steps += t.steps;
    cost[i] = 3 * ((t.H + hpw - 1) / hpw) + 4 * t.steps;  // head groups, and each step's start
  }
  if (bwd) {
    long long left = slots;
    int b0 = 0;
    for (int i = 0; i < p->n_parts; ++i) {
      RopePart& t = p->part[i];
      long long nb = part_blocks(*p, i, slots, cost, left);
      left -= nb;
      plan_tasks(p->tokens, t.steps, nb * rp::WARPS, 16, &t.spt, &t.cpt);
      const long long need = ((long long)p->tokens * t.cpt + rp::WARPS - 1) / rp::WARPS;
      if (nb > need) nb = need;
      t.b0 = b0;
      t.nb = (int)nb;
      b0 += t.nb;
    }
    return b0;
  }
  p->steps = (int)steps;
  plan_tasks(p->tokens, p->steps, slots * rp::WARPS, 8, &p->spt, &p->cpt);
  const long long need = ((long long)p->tokens * p->cpt + rp::WARPS - 1) / rp::WARPS;
  return (int)(need < slots ? need : slots);
}

template <typename... Args>
static cudaError_t launch_pdl(void (*kernel)(Args...), dim3 grid, int threads, int smem,
                              cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// kind: 0 contiguous outputs, 1 pages, 2 gradient.
template <int D, typename T>
static int launch_rope_t(const RopeParams& p, int blocks, int kind, bool il, bool few,
                         cudaStream_t s) {
  void (*const kernels[12])(RopeParams) = {
      rope_kernel<D, T, false, false>,     rope_kernel<D, T, true, false>,
      rope_kernel<D, T, false, true>,      rope_kernel<D, T, true, true>,
      rope_bwd_kernel<D, T, false, false>, rope_bwd_kernel<D, T, true, false>,
      rope_few_kernel<D, T, false, false>, rope_few_kernel<D, T, true, false>,
      rope_few_kernel<D, T, false, true>,  rope_few_kernel<D, T, true, true>,
      rope_bwd_kernel<D, T, false, true>,  rope_bwd_kernel<D, T, true, true>};
  auto smem = [](int k) {
    return k < 4 ? rp::Cfg<D, false>::SMEM_TOTAL
           : k < 6 ? rp::Cfg<D, true>::SMEM_TOTAL
           : k < 10 ? rp::Cfg<D, false, true>::SMEM_TOTAL : rp::Cfg<D, true, true>::SMEM_TOTAL;
  };
  static int attr_set[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE)) {
    for (int k = 0; k < 12; ++k) {
      e = cudaFuncSetAttribute(kernels[k], cudaFuncAttributeMaxDynamicSharedMemorySize, smem(k));
      if (e != cudaSuccess) return e;
    }
    if (dev >= 0 && dev < 64) __atomic_store_n(&attr_set[dev], 1, __ATOMIC_RELEASE);
  }
  const int k = 6 * (few ? 1 : 0) + 2 * kind + (il ? 1 : 0);
  return launch_pdl(kernels[k], dim3(blocks), rp::THREADS, smem(k), s, p);
}

static int launch_rope(const RopeParams& p, int blocks, int D, bool bf16, int kind, bool il,
                       bool few, cudaStream_t s) {
  if (D == 64)
    return bf16 ? launch_rope_t<64, __nv_bfloat16>(p, blocks, kind, il, few, s)
                : launch_rope_t<64, __half>(p, blocks, kind, il, few, s);
  return bf16 ? launch_rope_t<128, __nv_bfloat16>(p, blocks, kind, il, few, s)
              : launch_rope_t<128, __half>(p, blocks, kind, il, few, s);
}

int set_rope_wait_limit(unsigned long long ns) { return set_wait_limit_this_unit(ns); }

int read_rope_error(unsigned int* out, int reset) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_rope_err, sizeof(v));
  if (e != cudaSuccess) return e;
  if (reset && v) {
    const unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_rope_err, &z, sizeof(z));
    if (e != cudaSuccess) return e;
  }
  *out = v;
  return cudaSuccess;
}

}  // namespace fa

namespace {

bool al(const void* p, unsigned n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Rules shared by the three entry points.
bool rope_sizes_ok(long long T, int Hq, int Hkv, int D, int rot, float eps, int dtype) {
  if (T < 0 || Hq < 0 || Hkv < 0) return false;
  if (D != 64 && D != 128) return false;
  if (rot < 16 || rot > D || rot % 16 != 0) return false;
  if (!isfinite(eps) || !(eps > 0.f)) return false;
  if (dtype != FA_BF16 && dtype != FA_FP16) return false;
  // Token indexes fit 31 bits with room for the warps' stride.
  if (T > INT32_MAX - (1 << 20) || Hq > (1 << 20) || Hkv > (1 << 20)) return false;
  return true;
}

// x: [tokens][H][D] with the given token stride in elements.
bool heads_ok(const void* x, long long stride, int H, int D) {
  return al(x, 16) && stride % 8 == 0 && stride >= (long long)H * D && stride < (1ll << 40);
}

fa::RopePart part(const void* x, long long xs, int H, const void* w, void* y, const void* g,
                  bool paged) {
  fa::RopePart t = {};
  t.x = x;
  t.xs = xs;
  t.H = H;
  t.w = w;
  t.y = y;
  t.g = g;
  t.paged = paged ? 1 : 0;
  return t;
}

}  // namespace

extern "C" int fa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out,
                               const void* q_weight, const void* k_weight, const float* inv_freq,
                               const int32_t* positions, long long T, int Hq, int Hkv, int D,
                               int rot_dim, long long q_stride, long long k_stride, float eps,
                               int interleaved, int dtype, cudaStream_t stream) {
  if (!rope_sizes_ok(T, Hq, Hkv, D, rot_dim, eps, dtype)) return FA_ERR_INVALID_ARG;
  if (T == 0 || (Hq == 0 && Hkv == 0)) return FA_OK;
  if (!al(inv_freq, 4) || !al(positions, 4)) return FA_ERR_INVALID_ARG;
  if (Hq && (!heads_ok(q, q_stride, Hq, D) || !al(q_out, 16) || !al(q_weight, 16)))
    return FA_ERR_INVALID_ARG;
  if (Hkv && (!heads_ok(k, k_stride, Hkv, D) || !al(k_out, 16) || !al(k_weight, 16)))
    return FA_ERR_INVALID_ARG;
  const fa::SetupDuringCapture setup;
  fa::RopeParams p = {};
  if (Hq) p.part[p.n_parts++] = part(q, q_stride, Hq, q_weight, q_out, nullptr, false);
  if (Hkv) p.part[p.n_parts++] = part(k, k_stride, Hkv, k_weight, k_out, nullptr, false);
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.tokens = (int)T;
  p.rot = rot_dim;
  p.eps = eps;
  bool few;
  const int blocks = fa::plan_parts(&p, D, false, &few);
  return fa::record_cuda_status(
      fa::launch_rope(p, blocks, D, dtype == FA_BF16, 0, interleaved != 0, few, stream),
      "norm and rotation launch");
}

extern "C" int fa_qk_norm_rope_append(const void* q, const void* k, const void* v, void* q_out,
                                      void* kpages, void* vpages, const void* q_weight,
                                      const void* k_weight, const float* inv_freq,
                                      const int32_t* positions, const int32_t* page_table,
                                      const int32_t* seqlens, int B, int N, int Hq, int Hkv,
                                      int num_pages, int page_size, int max_pages, int D,
                                      int rot_dim, long long q_stride, long long k_stride,
                                      long long v_stride, float eps, int interleaved, int dtype,
                                      cudaStream_t stream) {
  if (B < 0 || N < 0 || num_pages < 0 || max_pages < 0) return FA_ERR_INVALID_ARG;
  if (!rope_sizes_ok((long long)B * N, Hq, Hkv, D, rot_dim, eps, dtype)) return FA_ERR_INVALID_ARG;
  if (page_size < 32 || page_size % 32 != 0) return FA_ERR_INVALID_ARG;
  if ((int64_t)max_pages * page_size > INT32_MAX) return FA_ERR_INVALID_ARG;
  if (B == 0 || N == 0 || (Hq == 0 && Hkv == 0)) return FA_OK;
  if (!al(inv_freq, 4) || !al(seqlens, 4) || (positions && !al(positions, 4)))
    return FA_ERR_INVALID_ARG;
  if (max_pages > 0 && !al(page_table, 4)) return FA_ERR_INVALID_ARG;
  if (Hq && (!heads_ok(q, q_stride, Hq, D) || !al(q_out, 16) || !al(q_weight, 16)))
    return FA_ERR_INVALID_ARG;
  if (Hkv && (!heads_ok(k, k_stride, Hkv, D) || !heads_ok(v, v_stride, Hkv, D) ||
              !al(k_weight, 16) || (num_pages > 0 && (!al(kpages, 16) || !al(vpages, 16)))))
    return FA_ERR_INVALID_ARG;
  if ((int64_t)num_pages * page_size > (1ll << 40) / (2 * D) / (Hkv ? Hkv : 1))
    return FA_ERR_INVALID_ARG;
  const fa::SetupDuringCapture setup;
  fa::RopeParams p = {};
  if (Hq) p.part[p.n_parts++] = part(q, q_stride, Hq, q_weight, q_out, nullptr, false);
  if (Hkv) {
    p.part[p.n_parts++] = part(k, k_stride, Hkv, k_weight, kpages, nullptr, true);
    p.part[p.n_parts++] = part(v, v_stride, Hkv, nullptr, vpages, nullptr, true);
  }
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.page_table = page_table;
  p.seqlens = seqlens;
  p.N = N;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.tokens = B * N;
  p.rot = rot_dim;
  p.eps = eps;
  bool few;
  const int blocks = fa::plan_parts(&p, D, false, &few);
  return fa::record_cuda_status(
      fa::launch_rope(p, blocks, D, dtype == FA_BF16, 1, interleaved != 0, few, stream),
      "norm, rotation and append launch");
}

extern "C" int fa_qk_norm_rope_backward(const void* dq_out, const void* dk_out, const void* q,
                                        const void* k, const void* q_weight, const void* k_weight,
                                        const float* inv_freq, const int32_t* positions, void* dq,
                                        void* dk, float* dq_weight, float* dk_weight, long long T,
                                        int Hq, int Hkv, int D, int rot_dim, long long q_stride,
                                        long long k_stride, float eps, int interleaved, int dtype,
                                        cudaStream_t stream) {
  if (!rope_sizes_ok(T, Hq, Hkv, D, rot_dim, eps, dtype)) return FA_ERR_INVALID_ARG;
  if (!al(dq_weight, 4) || !al(dk_weight, 4)) return FA_ERR_INVALID_ARG;
  if (T > 0 && (Hq || Hkv) && (!al(inv_freq, 4) || !al(positions, 4))) return FA_ERR_INVALID_ARG;
  if (T > 0 && Hq &&
      (!heads_ok(q, q_stride, Hq, D) || !al(dq_out, 16) || !al(dq, 16) || !al(q_weight, 16)))
    return FA_ERR_INVALID_ARG;
  if (T > 0 && Hkv &&
      (!heads_ok(k, k_stride, Hkv, D) || !al(dk_out, 16) || !al(dk, 16) || !al(k_weight, 16)))
    return FA_ERR_INVALID_ARG;
  // A side without rows has a zero weight gradient.
  cudaError_t e = cudaSuccess;
  if (T == 0 || Hq == 0) e = cudaMemsetAsync(dq_weight, 0, D * sizeof(float), stream);
  if (e == cudaSuccess && (T == 0 || Hkv == 0))
    e = cudaMemsetAsync(dk_weight, 0, D * sizeof(float), stream);
  if (e != cudaSuccess || T == 0 || (Hq == 0 && Hkv == 0))
    return fa::record_cuda_status(e, "norm and rotation gradient zero-fill");
  const fa::SetupDuringCapture setup;
  fa::RopeParams p = {};
  int iq = -1, ik = -1;
  if (Hq) {
    iq = p.n_parts;
    p.part[p.n_parts++] = part(q, q_stride, Hq, q_weight, dq, dq_out, false);
  }
  if (Hkv) {
    ik = p.n_parts;
    p.part[p.n_parts++] = part(k, k_stride, Hkv, k_weight, dk, dk_out, false);
  }
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.tokens = (int)T;
  p.rot = rot_dim;
  p.eps = eps;
  bool few;
  const int blocks = fa::plan_parts(&p, D, true, &few);
  void* scratch = nullptr;
  e = fa::scratch_alloc(&scratch, (size_t)blocks * D * sizeof(float), stream);
  if (e != cudaSuccess) return fa::record_cuda_status(e, "norm and rotation gradient scratch");
  p.partial = static_cast<float*>(scratch);
  int r = fa::launch_rope(p, blocks, D, dtype == FA_BF16, 2, interleaved != 0, few, stream);
  if (r == 0)
    r = fa::launch_pdl(fa::rope_dw_kernel, dim3(D / 32, 2), fa::kDwThreads, 0, stream,
                       (const float*)p.partial, D, iq >= 0 ? p.part[iq].b0 : 0,
                       iq >= 0 ? p.part[iq].nb : 0, iq >= 0 ? dq_weight : (float*)nullptr,
                       ik >= 0 ? p.part[ik].b0 : 0, ik >= 0 ? p.part[ik].nb : 0,
                       ik >= 0 ? dk_weight : (float*)nullptr);
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  if (r != 0) return fa::record_cuda_status(r, "norm and rotation gradient launch");
  return fa::record_cuda_status(ef, "norm and rotation gradient cudaFreeAsync");
}
