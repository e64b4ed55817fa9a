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
// one token.  A warp keeps one token's cosines and sines in registers over
// all of that token's heads that it takes.
//
// Angles: positions reach 2^31, where an fp32 product p * inv_freq has no
// correct bit left.  Each block turns inv_freq once into a 64-bit fixed-point
// fraction of a turn; the phase p * fraction is then an integer product
// modulo 2^64 (whole turns drop out by overflow), good to about 2^-25 turns at
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
constexpr int UNR = 2;  // head groups per step; a step's loads run ahead by one step
constexpr int BLOCKS_PER_SM = 2;
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

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = unpack2<T>(w[j]);
    f[2 * j] = v.x;
    f[2 * j + 1] = v.y;
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                    pack2<T>(f[6], f[7]));
}

// One of the tensors a launch walks: queries, keys or values.
struct RopePart {
  const void* x;  // [tokens][H][D], token stride xs elements
  const void* g;  // gradient: dL/dout, contiguous
  void* y;        // contiguous output, or pages
  const void* w;  // [D]; null: copy the heads as they are (values)
  long long xs;
  int H;
  int paged;
  // Forward: the part's head groups are [first, first + units) of a token's.
  int first, units;
  // Gradient: blocks [b0, b0 + nb) of the grid walk the part.
  int b0, nb;
  // A task is up to upt head groups of one token, cpt tasks per token.
  int upt, cpt;
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
  long long tokens;
  int groups, upt, cpt;  // forward: head groups of a token, and its tasks
  int rot;
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

template <int D, bool IL>
__device__ __forceinline__ void cos_sin(const LaneMap<D, IL>& m, int rot, int pos,
                                        const unsigned long long* sF, float (&cs)[8],
                                        float (&sn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int f = m.freq(e, rot);
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (f >= 0) {
      const unsigned long long ph = sF[f] * (unsigned long long)(long long)pos;
      // Signed fraction of a turn in [-1/2, 1/2), times two: half turns.
      sincospif(__ll2float_rn((long long)ph) * 1.0842021724855044e-19f, &sn[e], &cs[e]);
    }
  }
}

// Pair e of a lane's 16 elements, as (first, second).
template <bool IL>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&cs)[8],
                                     const float (&sn)[8], float sign) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float s = sign * sn[e];
    if constexpr (IL) {
      float(&v)[8] = e < 4 ? a : b;
      const int k = 2 * (e & 3);
      const float p = v[k], q = v[k + 1];
      v[k] = p * cs[e] - q * s;
      v[k + 1] = q * cs[e] + p * s;
    } else {
      const float p = a[e], q = b[e];
      a[e] = p * cs[e] - q * s;
      b[e] = q * cs[e] + p * s;
    }
  }
}

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A warp's place in its tasks: warps take tasks in a grid stride, a step at a
// time.  (The stride is added as whole tokens and tasks: no division per task.)
struct RopeWalk {
  long long t;  // token
  int c;        // task of the token
  int u;        // head group
  __device__ __forceinline__ RopeWalk(long long w, int cpt, int upt) {
    t = w / cpt;
    c = (int)(w - t * cpt);
    u = c * upt;
  }
  __device__ __forceinline__ int end(int upt, int groups) const {
    const int e = (c + 1) * upt;
    return e < groups ? e : groups;
  }
  __device__ __forceinline__ void next_task(int cpt, int upt, long long dt, int dc) {
    t += dt;
    c += dc;
    if (c >= cpt) {
      c -= cpt;
      ++t;
    }
    u = c * upt;
  }
};

// Cache row of token t (slot seqlens[b] - N + s), in rows of the pool, or -1
// (a padding sequence, or a length or page id out of range, which sets the
// bounds bit); *slot receives the position in the sequence.
__device__ __forceinline__ long long cache_row(const RopeParams& p, long long t, int* slot) {
  const int b = (int)(t / p.N), s = (int)(t - (long long)b * p.N);
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

// HPW heads of one token make a head group; a token's groups are its query
// heads', then its keys', then (paged) its values'.  Each warp keeps one step of
// UNR groups in registers while the next step's loads are on their way, across
// the ends of its tasks too.
template <int D, typename T, bool IL, bool PAGED>
__global__ void __launch_bounds__(rp::THREADS, rp::BLOCKS_PER_SM)
    rope_kernel(const __grid_constant__ RopeParams p) {
  using M = LaneMap<D, IL>;
  __shared__ unsigned long long sF[D / 2];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31;
  const M m(lane, p.rot);
  const long long warps = (long long)gridDim.x * rp::WARPS;
  const long long w0 = (long long)blockIdx.x * rp::WARPS + (threadIdx.x >> 5);
  const long long dt = warps / p.cpt;
  const int dc = (int)(warps - dt * p.cpt);
  RopeWalk at(w0, p.cpt, p.upt);

  // The part of head group u.
  auto part_of = [&](int u) {
    int i = 0;
    if (p.n_parts > 1 && u >= p.part[1].first) i = 1;
    if (PAGED && p.n_parts > 2 && u >= p.part[2].first) i = 2;
    return i;
  };
  auto load = [&](const RopeWalk& a, uint4 (&r)[rp::UNR][2], int* pos) {
    if (a.t >= p.tokens) return;
    const int end = a.end(p.upt, p.groups);
#pragma unroll
    for (int j = 0; j < rp::UNR; ++j) {
      const int u = a.u + j;
      if (u < end) {
        const RopePart& pt = p.part[part_of(u)];
        const int h = (u - pt.first) * M::HPW + m.sub;
        if (h < pt.H) {
          const T* x = static_cast<const T*>(pt.x) + a.t * pt.xs + (size_t)h * D;
          r[j][0] = *reinterpret_cast<const uint4*>(x + m.c0 * 8);
          r[j][1] = *reinterpret_cast<const uint4*>(x + m.c1 * 8);
        }
      }
    }
    if (!PAGED || p.positions) *pos = p.positions[a.t];
  };

  uint4 cur[rp::UNR][2], nxt[rp::UNR][2];
#pragma unroll
  for (int j = 0; j < rp::UNR; ++j)
    cur[j][0] = cur[j][1] = nxt[j][0] = nxt[j][1] = make_uint4(0u, 0u, 0u, 0u);
  int pos = 0, pos_n = 0;
  load(at, cur, &pos);
  load_fractions(p.inv_freq, p.rot / 2, sF);
  long long token = -1, row = 0;
  int kind = -1;
  float cs[8], sn[8];
  uint4 wa = make_uint4(0u, 0u, 0u, 0u), wb = wa;
  while (at.t < p.tokens) {
    RopeWalk nx = at;
    nx.u += rp::UNR;
    if (nx.u >= at.end(p.upt, p.groups)) nx.next_task(p.cpt, p.upt, dt, dc);
    load(nx, nxt, &pos_n);
    if (at.t != token) {  // warp-uniform, as is every branch on the walk
      token = at.t;
      if constexpr (PAGED) {
        int slot;
        row = cache_row(p, token, &slot);
        if (!p.positions) pos = slot;
      }
      cos_sin<D, IL>(m, p.rot, pos, sF, cs, sn);
    }
    const int end = at.end(p.upt, p.groups);
#pragma unroll
    for (int j = 0; j < rp::UNR; ++j) {
      const int u = at.u + j;
      if (u >= end) break;
      const int i = part_of(u);
      const RopePart& pt = p.part[i];
      const int h = (u - pt.first) * M::HPW + m.sub;
      const bool norm = !PAGED || pt.w != nullptr;
      if (i != kind) {
        kind = i;
        if (norm) {
          wa = *reinterpret_cast<const uint4*>(static_cast<const T*>(pt.w) + m.c0 * 8);
          wb = *reinterpret_cast<const uint4*>(static_cast<const T*>(pt.w) + m.c1 * 8);
        }
      }
      if (norm) {
        float a[8], b[8], w[8];
        unpack8<T>(cur[j][0], a);
        unpack8<T>(cur[j][1], b);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
        ss = head_sum<M::LPH>(ss);
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        unpack8<T>(wa, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] *= r * w[e];
        unpack8<T>(wb, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] *= r * w[e];
        turn<IL>(a, b, cs, sn, 1.f);
        cur[j][0] = pack8<T>(a);
        cur[j][1] = pack8<T>(b);
      }
      const long long to = PAGED && pt.paged ? row : token;
      if (h < pt.H && (!PAGED || to >= 0)) {
        T* y = static_cast<T*>(pt.y) + (to * pt.H + h) * D;
        *reinterpret_cast<uint4*>(y + m.c0 * 8) = cur[j][0];
        *reinterpret_cast<uint4*>(y + m.c1 * 8) = cur[j][1];
      }
    }
    at = nx;
    pos = pos_n;
#pragma unroll
    for (int j = 0; j < rp::UNR; ++j) {
      cur[j][0] = nxt[j][0];
      cur[j][1] = nxt[j][1];
    }
  }
}

// Gradient of rope_kernel.  Each block walks the queries or the keys, a head
// group per step with the next step's loads ahead, and ends with one row of
// partial[] (its sum of gy x r per column); the sums of a lane, a block and the
// blocks are taken in a fixed order, so equal calls give equal bits.
template <int D, typename T, bool IL>
__global__ void __launch_bounds__(rp::THREADS, rp::BLOCKS_PER_SM)
    rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  using M = LaneMap<D, IL>;
  __shared__ unsigned long long sF[D / 2];
  __shared__ float sW[rp::WARPS][D];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const M m(lane, p.rot);
  const RopePart& pt = p.part[p.n_parts > 1 && (int)blockIdx.x >= p.part[1].b0 ? 1 : 0];
  const T* x = static_cast<const T*>(pt.x);
  const T* g = static_cast<const T*>(pt.g);
  T* dx = static_cast<T*>(pt.y);
  const long long warps = (long long)pt.nb * rp::WARPS;
  const long long dt = warps / pt.cpt;
  const int dc = (int)(warps - dt * pt.cpt);
  RopeWalk at((long long)(blockIdx.x - pt.b0) * rp::WARPS + warp, pt.cpt, pt.upt);

  auto load = [&](const RopeWalk& q, uint4 (&r)[4], int* pos) {
    const int h = q.u * M::HPW + m.sub;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = make_uint4(0u, 0u, 0u, 0u);
    if (q.t >= p.tokens) return;
    if (h < pt.H) {
      const T* xt = x + q.t * pt.xs + (size_t)h * D;
      const T* gt = g + (q.t * pt.H + h) * D;
      r[0] = *reinterpret_cast<const uint4*>(xt + m.c0 * 8);
      r[1] = *reinterpret_cast<const uint4*>(xt + m.c1 * 8);
      r[2] = *reinterpret_cast<const uint4*>(gt + m.c0 * 8);
      r[3] = *reinterpret_cast<const uint4*>(gt + m.c1 * 8);
    }
    *pos = p.positions[q.t];
  };
  uint4 cur[4], nxt[4];
  int pos = 0, pos_n = 0;
  load(at, cur, &pos);
  const uint4 wa = *reinterpret_cast<const uint4*>(static_cast<const T*>(pt.w) + m.c0 * 8);
  const uint4 wb = *reinterpret_cast<const uint4*>(static_cast<const T*>(pt.w) + m.c1 * 8);
  load_fractions(p.inv_freq, p.rot / 2, sF);
  float acc0[8], acc1[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc0[e] = acc1[e] = 0.f;
  long long token = -1;
  float cs[8], sn[8];
  while (at.t < p.tokens) {
    RopeWalk nx = at;
    if (++nx.u >= at.end(pt.upt, pt.units)) nx.next_task(pt.cpt, pt.upt, dt, dc);
    load(nx, nxt, &pos_n);
    const int h = at.u * M::HPW + m.sub;
    float a[8], b[8], ga[8], gb[8], w[8];
    if (at.t != token) {
      token = at.t;
      cos_sin<D, IL>(m, p.rot, pos, sF, cs, sn);
    }
    unpack8<T>(cur[2], ga);
    unpack8<T>(cur[3], gb);
    turn<IL>(ga, gb, cs, sn, -1.f);
    unpack8<T>(cur[0], a);
    unpack8<T>(cur[1], b);
    float ss = 0.f, dot = 0.f;
    unpack8<T>(wa, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ss += a[e] * a[e] + b[e] * b[e];
      dot += a[e] * (w[e] * ga[e]);
    }
    unpack8<T>(wb, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) dot += b[e] * (w[e] * gb[e]);
    ss = head_sum<M::LPH>(ss);
    dot = head_sum<M::LPH>(dot);
    const float r = rsqrtf(ss * (1.f / D) + p.eps);
    const float f = dot * (1.f / D) * r * r;  // r^2 mean(x w gy)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc0[e] += ga[e] * (a[e] * r);
      acc1[e] += gb[e] * (b[e] * r);
      b[e] = r * (w[e] * gb[e] - b[e] * f);
    }
    unpack8<T>(wa, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = r * (w[e] * ga[e] - a[e] * f);
    if (h < pt.H) {
      T* d = dx + (token * pt.H + h) * D;
      *reinterpret_cast<uint4*>(d + m.c0 * 8) = pack8<T>(a);
      *reinterpret_cast<uint4*>(d + m.c1 * 8) = pack8<T>(b);
    }
    at = nx;
    pos = pos_n;
#pragma unroll
    for (int e = 0; e < 4; ++e) cur[e] = nxt[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = M::LPH; o < 32; o <<= 1) {  // the lanes of the warp's other heads
      acc0[e] += __shfl_xor_sync(0xffffffffu, acc0[e], o);
      acc1[e] += __shfl_xor_sync(0xffffffffu, acc1[e], o);
    }
    if (m.sub == 0) {
      sW[warp][m.c0 * 8 + e] = acc0[e];
      sW[warp][m.c1 * 8 + e] = acc1[e];
    }
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < rp::WARPS; ++i) s += sW[i][threadIdx.x];
    p.partial[(size_t)blockIdx.x * D + threadIdx.x] = s;
  }
}

// dw of part blockIdx.y: the sum of its blocks' partial rows, 32 columns per
// block, 8 interleaved row sums each.
__global__ void __launch_bounds__(256)
    rope_dw_kernel(const float* partial, int D, int b0q, int nbq, float* dqw, int b0k, int nbk,
                   float* dkw) {
  __shared__ float sS[8][32];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int b0 = blockIdx.y ? b0k : b0q, nb = blockIdx.y ? nbk : nbq;
  float* dw = blockIdx.y ? dkw : dqw;
  if (!dw) return;
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  float s = 0.f;
#pragma unroll 4
  for (int i = r; i < nb; i += 8) s += partial[(size_t)(b0 + i) * D + col];
  sS[r][c] = s;
  __syncthreads();
  if (r == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sS[i][c];
    dw[col] = s;
  }
}

// Head groups per task: the fewest rounds of the resident warps, a round
// costing its groups and, once, the token's cosines and sines (about as much
// as two groups).
static void plan_tasks(long long tokens, int groups, long long warps, int* upt, int* cpt) {
  long long best = 0;
  for (int c = 1; c <= groups && c <= 64; ++c) {
    const int u = (groups + c - 1) / c;
    if ((groups + u - 1) / u != c) continue;
    const long long cost = (tokens * c + warps - 1) / warps * (u + 2);
    if (best == 0 || cost < best) {
      best = cost;
      *upt = u;
      *cpt = c;
    }
  }
}

// Head groups, tasks and blocks.  Returns the grid size.
static int plan_parts(RopeParams* p, int D, bool bwd) {
  const int hpw = 32 / (D / 16);
  const int sms = sm_count() > 0 ? sm_count() : 148;
  const long long slots = (long long)sms * rp::BLOCKS_PER_SM;  // resident blocks
  long long groups = 0;
  for (int i = 0; i < p->n_parts; ++i) {
    RopePart& t = p->part[i];
    t.units = (t.H + hpw - 1) / hpw;
    t.first = (int)groups;
    groups += t.units;
  }
  if (bwd) {
    // Blocks in proportion to the parts' head groups, all resident at once.
    long long left = slots;
    int b0 = 0;
    for (int i = 0; i < p->n_parts; ++i) {
      RopePart& t = p->part[i];
      long long nb = i + 1 < p->n_parts ? (slots * t.units + groups / 2) / groups : left;
      if (nb > left - (p->n_parts - 1 - i)) nb = left - (p->n_parts - 1 - i);
      if (nb < 1) nb = 1;
      left -= nb;
      plan_tasks(p->tokens, t.units, nb * rp::WARPS, &t.upt, &t.cpt);
      const long long need = (p->tokens * t.cpt + rp::WARPS - 1) / rp::WARPS;
      if (nb > need) nb = need;
      t.b0 = b0;
      t.nb = (int)nb;
      b0 += t.nb;
    }
    return b0;
  }
  p->groups = (int)groups;
  plan_tasks(p->tokens, p->groups, slots * rp::WARPS, &p->upt, &p->cpt);
  const long long need = (p->tokens * p->cpt + rp::WARPS - 1) / rp::WARPS;
  return (int)(need < slots ? need : slots);
}

template <typename... Args>
static cudaError_t launch_pdl(void (*kernel)(Args...), dim3 grid, int threads,
                              cudaStream_t stream, Args... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, typename T>
static int launch_rope_t(const RopeParams& p, int blocks, bool paged, bool bwd, bool il,
                         cudaStream_t s) {
  if (bwd)
    return il ? launch_pdl(rope_bwd_kernel<D, T, true>, dim3(blocks), rp::THREADS, s, p)
              : launch_pdl(rope_bwd_kernel<D, T, false>, dim3(blocks), rp::THREADS, s, p);
  if (paged)
    return il ? launch_pdl(rope_kernel<D, T, true, true>, dim3(blocks), rp::THREADS, s, p)
              : launch_pdl(rope_kernel<D, T, false, true>, dim3(blocks), rp::THREADS, s, p);
  return il ? launch_pdl(rope_kernel<D, T, true, false>, dim3(blocks), rp::THREADS, s, p)
            : launch_pdl(rope_kernel<D, T, false, false>, dim3(blocks), rp::THREADS, s, p);
}

static int launch_rope(const RopeParams& p, int blocks, int D, bool bf16, bool paged, bool bwd,
                       bool il, cudaStream_t s) {
  if (D == 64)
    return bf16 ? launch_rope_t<64, __nv_bfloat16>(p, blocks, paged, bwd, il, s)
                : launch_rope_t<64, __half>(p, blocks, paged, bwd, il, s);
  return bf16 ? launch_rope_t<128, __nv_bfloat16>(p, blocks, paged, bwd, il, s)
              : launch_rope_t<128, __half>(p, blocks, paged, bwd, il, s);
}

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
  // Work indexes (tasks) and element offsets stay far inside 63 bits.
  if (T > (1ll << 40) || Hq > (1 << 20) || Hkv > (1 << 20)) return false;
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
  fa::RopeParams p = {};
  if (Hq) p.part[p.n_parts++] = part(q, q_stride, Hq, q_weight, q_out, nullptr, false);
  if (Hkv) p.part[p.n_parts++] = part(k, k_stride, Hkv, k_weight, k_out, nullptr, false);
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.tokens = T;
  p.rot = rot_dim;
  p.eps = eps;
  const int blocks = fa::plan_parts(&p, D, false);
  return fa::record_cuda_status(
      fa::launch_rope(p, blocks, D, dtype == FA_BF16, false, false, interleaved != 0, stream),
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
  p.tokens = (long long)B * N;
  p.rot = rot_dim;
  p.eps = eps;
  const int blocks = fa::plan_parts(&p, D, false);
  return fa::record_cuda_status(
      fa::launch_rope(p, blocks, D, dtype == FA_BF16, true, false, interleaved != 0, stream),
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
  p.tokens = T;
  p.rot = rot_dim;
  p.eps = eps;
  const int blocks = fa::plan_parts(&p, D, true);
  void* scratch = nullptr;
  e = fa::scratch_alloc(&scratch, (size_t)blocks * D * sizeof(float), stream);
  if (e != cudaSuccess) return fa::record_cuda_status(e, "norm and rotation gradient scratch");
  p.partial = static_cast<float*>(scratch);
  int r = fa::launch_rope(p, blocks, D, dtype == FA_BF16, false, true, interleaved != 0, stream);
  if (r == 0)
    r = fa::launch_pdl(fa::rope_dw_kernel, dim3(D / 32, 2), 256, stream,
                       (const float*)p.partial, D, iq >= 0 ? p.part[iq].b0 : 0,
                       iq >= 0 ? p.part[iq].nb : 0, iq >= 0 ? dq_weight : (float*)nullptr,
                       ik >= 0 ? p.part[ik].b0 : 0, ik >= 0 ? p.part[ik].nb : 0,
                       ik >= 0 ? dk_weight : (float*)nullptr);
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  if (r != 0) return fa::record_cuda_status(r, "norm and rotation gradient launch");
  return fa::record_cuda_status(ef, "norm and rotation gradient cudaFreeAsync");
}
