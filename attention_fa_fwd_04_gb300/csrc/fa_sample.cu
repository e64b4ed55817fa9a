// fa_sample.cu -- the next token of every row of logits: temperature, top-k,
// top-p, min-p and a given uniform number (fa_sample).
//
// With weights w_i = exp((l_i - max l) / T), tokens ordered by logit (equal ones by
// index):
//   top-k   keeps the first k of the order;
//   top-p   keeps, of those, the tokens before which less than p of their weight lies;
//   min-p   keeps w_i >= min_p (the largest weight is 1).
// Each keeps a beginning of the order, so what is kept is "logit above a border, and
// the first m of the tokens at the border".  The token is the lowest index whose
// cumulative kept weight (by index) exceeds u times all of it.
//
// Nothing is sorted.  The border is found by narrowing an interval of keys (the
// logits' bits, made to order as whole numbers): a pass over the row counts the
// keys of the interval in 2048 bins; for top-k the bin of the k-th is exact, for
// top-p the counts only suggest where the border is, and the next pass adds up the
// weights above and in the suggested bins exactly and goes on from what it finds.
//
// The answers are whole numbers.  With 128000 tokens an error of 1e-7 in the sums
// would move one draw in fifty, so weights are pairs of floats good to 2^-40
// (2^(j/256) from a table, the rest a short series), summed as pairs in a fixed
// order: about 40 fp32 operations per weight, where fp64 would be bound by the few
// fp64 units.
//
// Layout: a cluster of up to 8 CTAs takes a row and keeps it in shared memory, so
// that HBM is read once however many passes there are.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "fa.h"
#include "fa_exp2_table.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

namespace sa {
constexpr int CLUSTER = 8;
constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 2048;
constexpr int SEGS = CLUSTER * WARPS;  // index-ordered segments of a row, one per warp
constexpr int SMEM_MAX = 200 * 1024;   // bytes of a CTA's part of a row
}  // namespace sa

struct SampleParams {
  const void* logits;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* probs;  // [rows, V] or null
  long long stride;
  int V, cluster;
  int seg;  // elements per warp: whole steps of 32 groups
};

// 16 bytes of logits, and the logits' order as whole numbers (NaN counts as
// -infinity, -0 as 0).
template <typename T>
struct Logits;
template <>
struct Logits<float> {
  static constexpr int GROUP = 4, KEY_BITS = 32;
  typedef uint32_t raw;
  static __device__ __forceinline__ float value(raw r) { return __uint_as_float(r); }
  static __device__ __forceinline__ raw clean(raw r) {
    const float x = __uint_as_float(r);
    return x != x ? 0xff800000u : __float_as_uint(x + 0.f);
  }
  static __device__ __forceinline__ uint32_t key(raw r) {
    return r ^ (uint32_t)((int32_t)r >> 31 | (int32_t)0x80000000);
  }
  static __device__ __forceinline__ raw unkey(uint32_t k) {
    return k & 0x80000000u ? k ^ 0x80000000u : ~k;
  }
  static __device__ __forceinline__ raw at(const uint4& v, int e) {
    return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
  }
  static __device__ __forceinline__ raw from(float x) { return clean(__float_as_uint(x)); }
  // The lowest raw value that is at least x.
  static __device__ __forceinline__ raw at_least(double x) { return from(__double2float_ru(x)); }
};
template <typename H>
struct Logits16 {
  static constexpr int GROUP = 8, KEY_BITS = 16;
  typedef uint16_t raw;
  static __device__ __forceinline__ uint32_t key(raw r) {
    return r & 0x8000u ? (uint16_t)~r : (uint16_t)(r | 0x8000u);
  }
  static __device__ __forceinline__ raw unkey(uint32_t k) {
    return k & 0x8000u ? (raw)(k ^ 0x8000u) : (raw)~k;
  }
  static __device__ __forceinline__ raw at(const uint4& v, int e) {
    const uint32_t w = e < 2 ? v.x : e < 4 ? v.y : e < 6 ? v.z : v.w;
    return (raw)(e & 1 ? w >> 16 : w);
  }
};
template <>
struct Logits<__nv_bfloat16> : Logits16<__nv_bfloat16> {
  static __device__ __forceinline__ float value(raw r) { return __uint_as_float((uint32_t)r << 16); }
  static __device__ __forceinline__ raw clean(raw r) {
    return (r & 0x7fffu) > 0x7f80u ? (raw)0xff80u : (r == 0x8000u ? (raw)0 : r);
  }
  static __device__ __forceinline__ raw from(float x) {  // (rounds up)
    return clean(__bfloat16_as_ushort(__float2bfloat16_ru(x)));
  }
  static __device__ __forceinline__ raw at_least(double x) { return from(__double2float_ru(x)); }
};
template <>
struct Logits<__half> : Logits16<__half> {
  static __device__ __forceinline__ float value(raw r) { return __half2float(__ushort_as_half(r)); }
  static __device__ __forceinline__ raw clean(raw r) {
    return (r & 0x7fffu) > 0x7c00u ? (raw)0xfc00u : (r == 0x8000u ? (raw)0 : r);
  }
  static __device__ __forceinline__ raw from(float x) {  // (rounds up)
    return clean(__half_as_ushort(__float2half_ru(x)));
  }
  static __device__ __forceinline__ raw at_least(double x) { return from(__double2float_ru(x)); }
};

// Unevaluated sum of two floats.
struct __align__(8) Sum2 {
  float hi, lo;
};
__device__ __forceinline__ Sum2 sum_of(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Sum2 sum_of(Sum2 a, Sum2 b) {
  const Sum2 s = sum_of(a.hi, b.hi);
  const float l = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)), h = __fadd_rn(s.hi, l);
  return {h, __fsub_rn(l, __fsub_rn(h, s.hi))};
}
__device__ __forceinline__ Sum2 times(Sum2 a, float b) {
  const float h = __fmul_rn(a.hi, b), l = __fmaf_rn(a.lo, b, __fmaf_rn(a.hi, b, -h));
  const float s = __fadd_rn(h, l);
  return {s, __fsub_rn(l, __fsub_rn(s, h))};
}
__device__ __forceinline__ bool exceeds(Sum2 a, Sum2 b) {
  const Sum2 d = sum_of(a.hi, -b.hi);
  return __fadd_rn(d.hi, __fadd_rn(d.lo, __fsub_rn(a.lo, b.lo))) > 0.f;
}
__device__ __forceinline__ Sum2 shfl_xor(Sum2 a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
}
__device__ __forceinline__ Sum2 warp_sum(Sum2 a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = sum_of(a, shfl_xor(a, o));
  return a;
}
// Sums of the lanes up to this one.
__device__ __forceinline__ Sum2 warp_sums(Sum2 a) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sum2 y = {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
    if (lane >= o) a = sum_of(y, a);
  }
  return a;
}
__device__ __forceinline__ Sum2 lane_of(Sum2 a, int l) {
  return {__shfl_sync(0xffffffffu, a.hi, l), __shfl_sync(0xffffffffu, a.lo, l)};
}
// (Only in one thread or warp: the SM has two fp64 units.)
__device__ __forceinline__ double wide(Sum2 a) { return (double)a.hi + (double)a.lo; }

// Weights of a row's logits.
struct Weigher {
  float top;         // the largest logit
  float s_hi, s_lo;  // log2(e) / T
  const float2* table;
  // exp((l - top) / T) to about 2^-40 of itself; below 2^-120 it is 0.
  __device__ __forceinline__ Sum2 operator()(float l) const {
    const Sum2 d = sum_of(l, -top);
    const float y = __fmul_rn(d.hi, s_hi);
    const float y_lo = __fadd_rn(__fmaf_rn(d.hi, s_hi, -y),
                                 __fmaf_rn(d.hi, s_lo, __fmul_rn(d.lo, s_hi)));
    // y = k / 256 + r, |r| <= 2^-9.
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
    const float yc = fmaxf(y, -121.f);
    const float t = __fmaf_rn(yc, 256.f, kMagic);
    const int k = __float_as_int(t) - __float_as_int(kMagic);
    const float r = __fmaf_rn(__fsub_rn(t, kMagic), -0.00390625f, yc);
    // 2^(r + y_lo) - 1 = hi + lo.
    constexpr float L_hi = 0.693147182464599609375f, L_lo = -1.904654299958e-9f;  // ln 2
    constexpr float c2 = 0.240226506959100712f, c3 = 0.0555041086648215800f;  // ln2^2/2, ln2^3/6
    const float hi = __fmul_rn(r, L_hi);
    float lo = __fmaf_rn(r, L_hi, -hi);
    lo = __fmaf_rn(r, L_lo, lo);
    lo = __fmaf_rn(y_lo, L_hi, lo);
    const float a2 = __fadd_rn(r, y_lo);  // (r y_lo counts: 2^-28)
    lo = __fmaf_rn(__fmul_rn(a2, a2), __fmaf_rn(a2, c3, c2), lo);
    const float2 T = table[k & 255];
    // T (1 + hi + lo).
    const float m = __fmul_rn(T.x, hi);
    float e = __fmaf_rn(T.x, hi, -m);
    e = __fmaf_rn(T.x, lo, e);
    e = __fadd_rn(e, __fmaf_rn(T.y, hi, T.y));
    const float a = __fadd_rn(T.x, m);
    e = __fadd_rn(e, __fsub_rn(m, __fsub_rn(a, T.x)));
    const float f = __int_as_float(((k >> 8) + 127) << 23);
    // (l = top: exactly 1, also where both are infinite; l = -infinity has a y that
    // is not above -120, or NaN.)
    if (l == top) return Sum2{1.f, 0.f};
    return y > -120.f ? Sum2{__fmul_rn(a, f), __fmul_rn(e, f)} : Sum2{0.f, 0.f};
  }
};

__device__ __forceinline__ uint32_t remote(const void* local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(rank));
  return r;
}
__device__ __forceinline__ void put(uint32_t at, float a, float b) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ void put(uint32_t at, int a) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(a) : "memory");
}
__device__ __forceinline__ uint4 get4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

template <typename T>
__global__ void __launch_bounds__(sa::THREADS) sample_kernel(const __grid_constant__ SampleParams p) {
  using Lg = Logits<T>;
  using raw = typename Lg::raw;
  constexpr int GROUP = Lg::GROUP;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ float2 s_table[256];
  __shared__ __align__(16) uint32_t s_hist[2][sa::BINS];
  __shared__ float2 s_first[sa::SEGS];       // every warp's largest logit, smallest lane maximum
  __shared__ float2 s_warp[2][3][sa::SEGS];  // per round and quantity: every warp's sum
  __shared__ int s_cnt[sa::SEGS];
  __shared__ float2 s_steps[32];
  __shared__ uint32_t s_scan[sa::WARPS];
  __shared__ float s_fscan[sa::WARPS];
  __shared__ int s_i[4], s_cut[2];
  __shared__ uint32_t s_key[2];
  __shared__ float s_f[8];
  __shared__ double s_d[8];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int C = p.cluster;
  const int rank = C > 1 ? (int)(blockIdx.x % C) : 0;
  const long long row = blockIdx.x / C;
  const int n = p.seg * sa::WARPS;  // elements of this CTA's part, in places that begin at
                                    // the 16 bytes the row begins in
  const int segs = C * sa::WARPS, seg_id = rank * sa::WARPS + warp;
  pdl_launch_dependents();
  if (t < 256) s_table[t] = make_float2(kExp2Table[t][0], kExp2Table[t][1]);
  for (int i = t; i < 2 * sa::BINS; i += sa::THREADS) (&s_hist[0][0])[i] = 0;
  pdl_wait_primary();

  auto sync = [&] {  // the cluster's CTAs meet; what they stored is visible
    if (C > 1) {
      asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
      __syncthreads();
    }
  };
  // ---- the row into shared memory, its largest logit ----
  const T* const src = static_cast<const T*>(p.logits) + row * p.stride;
  const int lead = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  const long long first = (long long)rank * n;  // place of this part's first element
  uint4* const part = reinterpret_cast<uint4*>(smem_raw);
  const int g0 = warp * (p.seg / GROUP), g1 = g0 + p.seg / GROUP;  // this warp's groups
  const raw NEG = Lg::from(-INFINITY);
  float temp = p.temperature ? p.temperature[row] : 1.f;
  if (temp > 3.402823466e38f) temp = 3.402823466e38f;
  const bool greedy = !(temp > 0.f);
  float mx = -INFINITY;
#pragma unroll 4
  for (int g = g0 + lane; g < g1; g += 32) {
    const long long e0 = first + (long long)g * GROUP - lead;  // the group's first token
    alignas(16) raw v[GROUP];
    if (e0 >= 0 && e0 + GROUP <= p.V) {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(src + e0);
    } else {
#pragma unroll
      for (int e = 0; e < GROUP; ++e)
        v[e] = e0 + e >= 0 && e0 + e < p.V ? reinterpret_cast<const raw*>(src)[e0 + e] : NEG;
    }
#pragma unroll
    for (int e = 0; e < GROUP; ++e) {
      v[e] = Lg::clean(v[e]);
      mx = fmaxf(mx, Lg::value(v[e]));
    }
    part[g] = *reinterpret_cast<uint4*>(v);
  }
  {
    float hi = mx, lo = mx;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    if (lane < C) put(remote(&s_first[seg_id], lane), hi, lo);
  }
  if (t == 0) {
    const double s = fmin(1.4426950408889634 / (greedy ? 1.0 : (double)temp), 0x1p100);
    s_f[0] = (float)s;
    s_f[1] = (float)(s - (double)s_f[0]);
  }
  sync();
  float top = -INFINITY;
  for (int i = lane; i < segs; i += 32) top = fmaxf(top, s_first[i].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  Weigher weigh;
  weigh.top = top;
  weigh.table = s_table;
  weigh.s_hi = s_f[0];
  weigh.s_lo = s_f[1];

  // Of every element of this warp: f(place in the part, raw value).
  auto each = [&](auto&& f) {
    for (int g = g0 + lane; g < g1; g += 32) {
      const uint4 v = part[g];
#pragma unroll
      for (int e = 0; e < GROUP; ++e) f(g * GROUP + e, Lg::at(v, e));
    }
  };
  // Exchanges alternate between two buffers of bins and sums, so that one barrier
  // each does: a CTA fills a buffer again only after the barrier that the others
  // reach when they have read it.
  int round = 0;
  static_assert(sa::BINS == 4 * sa::THREADS, "four bins per thread");
  auto gather = [&](uint32_t (&h)[4]) {  // four bins of all CTAs together
    uint4 s = make_uint4(0, 0, 0, 0);
    for (int c = 0; c < C; ++c) {
      const uint4 v = C > 1 ? get4(remote(&s_hist[round & 1][4 * t], c))
                            : *reinterpret_cast<const uint4*>(&s_hist[round & 1][4 * t]);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    h[0] = s.x;
    h[1] = s.y;
    h[2] = s.z;
    h[3] = s.w;
    *reinterpret_cast<uint4*>(&s_hist[(round & 1) ^ 1][4 * t]) = make_uint4(0, 0, 0, 0);
  };
  // Sum of the block's values before this thread's; sums: one entry per warp.
  auto sum_before = [&](auto mine, auto* sums) {
    auto x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const auto y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    x -= mine;
    for (int i = 0; i < warp; ++i) x += sums[i];
    return x;
  };
  auto shift_of = [](uint32_t lo, uint32_t hi) { return max(0, 21 - __clz((int)(hi - lo))); };

  const bool alive = top != -INFINITY;
  const uint32_t kmax = Lg::key(Lg::from(top));
  // What is kept: keys above `border`, and the first `ties` (by index) of those at it.
  uint32_t border = 0;
  int ties = INT_MAX;
  bool limited = false;  // whether `ties` leaves any out
  const int k = p.top_k ? p.top_k[row] : 0;
  const float tp = p.top_p ? p.top_p[row] : 1.f;
  const float mp = p.min_p ? p.min_p[row] : 0.f;
  if (alive && (greedy || k == 1 || tp <= 0.f)) {
    border = kmax;
    ties = 1;
    limited = true;
  } else if (alive) {
    if (k > 0 && k < p.V) {
      // The k-th largest is at least the w-th largest of the warps' smallest lane
      // maxima, w = ceil(k / 32): 32 tokens of each of w warps are.
      uint32_t lo = Lg::key(NEG), hi = kmax;
      const int w = (k + 31) / 32;
      if (w <= segs) {
        if (t < segs) {
          const float mine = s_first[t].y;
          int above = 0;
          for (int i = 0; i < segs; ++i) {
            const float o = s_first[i].y;
            above += o > mine || (o == mine && i < t);
          }
          if (above == w - 1) s_key[0] = Lg::key(Lg::from(mine));
        }
        __syncthreads();
        lo = s_key[0];
      }
      int above = 0;
      for (;;) {
        const int shift = shift_of(lo, hi);
        const uint32_t span = hi - lo;
        uint32_t* const hist = s_hist[round & 1];
        each([&](int, raw r) {
          const uint32_t d = hi - Lg::key(r);
          if (d <= span) atomicAdd(&hist[d >> shift], 1u);
        });
        sync();
        uint32_t h[4];
        gather(h);
        ++round;
        uint32_t before = (uint32_t)above + sum_before(h[0] + h[1] + h[2] + h[3], s_scan);
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // the bin that the k-th falls into
          if (before < (uint32_t)k && (uint32_t)k <= before + h[e]) {
            s_i[0] = 4 * t + e;
            s_i[1] = (int)before;
            s_i[2] = (int)h[e];
          }
          before += h[e];
        }
        __syncthreads();
        const uint32_t b = (uint32_t)s_i[0];
        above = s_i[1];
        const int in = s_i[2];
        const uint32_t new_hi = hi - (b << shift), width = (1u << shift) - 1;
        lo = new_hi - lo > width ? new_hi - width : lo;
        hi = new_hi;
        if (lo == hi) {
          border = hi;
          ties = k - above;
          limited = in > ties;
          break;
        }
      }
      __syncthreads();
    }
    if (tp < 1.f) {
      // Keys in [elo, ehi] hold the border, or all that is kept is above them; s_d[0] is
      // the weight above.  Below elo come only, with top-k, the tokens at its border.
      const bool had_k = ties != INT_MAX;
      const uint32_t k_border = border;
      const int k_ties = ties;
      uint32_t elo = had_k ? border + 1 : Lg::key(NEG), ehi = kmax;
      uint32_t blo = elo, bhi = ehi;
      if (t == 0) {
        s_d[0] = 0.0;                                                              // above
        s_d[1] = -1.0;                                                             // the target
        s_d[2] = had_k ? wide(weigh(Lg::value(Lg::unkey(border)))) : 0.0;          // a tie's weight
      }
      if (!had_k) {
        // Where the border may be, from counts in 2048 bins of 1/64 of the
        // temperature: weights e^(-1/64) of one another.
        uint32_t* const hist = s_hist[round & 1];
        const float to_bin = weigh.s_hi * (64.f * 0.6931471805599453f);
        each([&](int, raw r) {
          const float d = (top - Lg::value(r)) * to_bin;
          if (d < (float)(sa::BINS - 1)) atomicAdd(&hist[(int)d], 1u);
        });
        sync();
        uint32_t h[4];
        gather(h);
        ++round;
        float m4[4], mine = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          m4[e] = (float)h[e] * __expf(-((float)(4 * t + e) + 0.5f) * (1.f / 64.f));
          mine += m4[e];
        }
        if (t == 0) {
          s_key[0] = elo;
          s_key[1] = ehi;
        }
        float before = sum_before(mine, s_fscan);
        float want = 0.f;
        for (int i = 0; i < sa::WARPS; ++i) want += s_fscan[i];
        want *= tp;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (before < want && want <= before + m4[e]) {
            // Two bins to either side; the next pass finds out whether that was enough.
            const int b = 4 * t + e;
            const float w = temp * (1.f / 64.f);
            s_key[0] = Lg::key(Lg::from(top - w * (float)(b + 3)));
            s_key[1] = Lg::key(Lg::from(top - w * (float)(b - 2)));
          }
          before += m4[e];
        }
        __syncthreads();
        bhi = min(max(s_key[1], elo), ehi);
        blo = min(max(s_key[0], elo), bhi);
      }
      enum { IN_TAIL, ABOVE, BELOW, INSIDE, DONE };
      int what = had_k && border == kmax ? IN_TAIL : INSIDE;
      if (what == IN_TAIL) __syncthreads();
      for (bool have_total = false; what != IN_TAIL && what != DONE; have_total = true) {
        const int shift = shift_of(blo, bhi);
        const uint32_t bspan = bhi - blo, espan = ehi - elo;
        uint32_t* const hist = s_hist[round & 1];
        Sum2 sum[3] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};  // above, in and below the bins
        each([&](int, raw r) {
          const uint32_t key = Lg::key(r);
          if (ehi - key > espan) return;
          const bool in = bhi - key <= bspan, over = key > bhi;
          if (in) atomicAdd(&hist[(bhi - key) >> shift], 1u);
          if (!have_total || in || over) {
            const Sum2 wt = weigh(Lg::value(r));
            if (in)
              sum[1] = sum_of(sum[1], wt);
            else if (over)
              sum[0] = sum_of(sum[0], wt);
            else
              sum[2] = sum_of(sum[2], wt);
          }
        });
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const Sum2 s = warp_sum(sum[q]);
          if (lane < C) put(remote(&s_warp[round & 1][q][seg_id], lane), s.hi, s.lo);
        }
        sync();
        uint32_t h[4];
        gather(h);
        if (warp < 3) {  // one warp for each sum
          Sum2 s{0.f, 0.f};
          for (int i = lane; i < segs; i += 32) {
            const float2 v = s_warp[round & 1][warp][i];
            s = sum_of(s, Sum2{v.x, v.y});
          }
          s = warp_sum(s);
          if (lane == 0) s_d[4 + warp] = wide(s);
        }
        ++round;
        // Counts times the weight in the middle of each bin suggest the next bins.
        float m4[4], mine = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t off = (uint32_t)(4 * t + e) << shift;
          m4[e] = 0.f;
          if (h[e])
            m4[e] = (float)h[e] *
                    weigh(Lg::value(Lg::unkey(bhi - min(off + ((1u << shift) >> 1), bspan)))).hi;
          mine += m4[e];
        }
        float before = sum_before(mine, s_fscan);  // (and s_d is there)
        if (t == 0) {
          if (!have_total) s_d[1] = (double)tp * (s_d[4] + s_d[5] + s_d[6] + s_d[2] * (had_k ? k_ties : 0));
          const double A = s_d[0] + s_d[4], target = s_d[1];
          int w = INSIDE;
          if (A >= target && bhi != ehi) {
            w = ABOVE;
          } else if (A + s_d[5] < target) {
            w = blo == elo ? IN_TAIL : BELOW;
            s_d[0] = A + s_d[5];
          } else {
            s_d[0] = A;
            if (blo == bhi) {
              w = DONE;
              const double m = ceil((target - A) / wide(weigh(Lg::value(Lg::unkey(blo)))));
              s_i[1] = m < 1.0 ? 1 : (m > (double)h[0] ? (int)h[0] : (int)m);
              s_i[2] = s_i[1] < (int)h[0];
            }
          }
          s_f[2] = (float)(target - A);
          s_i[0] = w;
          s_i[3] = (int)(bspan >> shift);
        }
        __syncthreads();
        what = s_i[0];
        if (what == ABOVE) {
          blo = elo = bhi + 1;
          bhi = ehi;
        } else if (what == BELOW) {
          bhi = ehi = blo - 1;
          blo = elo;
        } else if (what == DONE) {
          border = blo;
          ties = s_i[1];
          limited = s_i[2];
        } else if (what == INSIDE) {
          elo = blo;
          ehi = bhi;
          const float want = s_f[2];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (before < want && want <= before + m4[e]) s_i[3] = 4 * t + e;
            before += m4[e];
          }
          __syncthreads();
          // One bin to either side, or the one key.
          const uint32_t b = (uint32_t)s_i[3], side = shift > 0 ? 1u : 0u;
          const uint32_t o0 = (b > side ? b - side : 0u) << shift;
          const unsigned long long o1 = ((unsigned long long)(b + side + 1) << shift) - 1;
          blo = o1 >= bspan ? blo : ehi - (uint32_t)o1;
          bhi = ehi - min(o0, bspan);
          if (blo == elo && bhi == ehi && blo < bhi) blo = bhi - (bhi - blo) / 2;  // (few bins)
        }
        __syncthreads();
      }
      if (what == IN_TAIL && had_k) {  // among the tokens at top-k's border
        if (t == 0) {
          // (Nothing above it: the weights are all 1.)
          const double m = k_border == kmax ? ceil((double)tp * k_ties)
                                            : ceil((s_d[1] - s_d[0]) / s_d[2]);
          s_i[0] = m < 1.0 ? 1 : (m > (double)k_ties ? k_ties : (int)m);
        }
        __syncthreads();
        ties = s_i[0];
        limited = limited || ties < k_ties;
      }
    }
    if (mp > 0.f) {
      // w >= min_p: l >= top + T ln(min_p).
      if (t == 0)
        s_key[0] = top == INFINITY ? kmax
                                   : Lg::key(Lg::at_least(fmin((double)top, (double)top + (double)temp * log((double)mp))));
      __syncthreads();
      const uint32_t lowest = min(s_key[0], kmax);
      if (lowest > border) {
        border = lowest;
        ties = INT_MAX;
        limited = false;
      }
    }
  }
  // ---- ties by index: the place of the last one that is kept ----
  long long cut = LLONG_MAX;
  if (limited) {
    int c = 0;
    each([&](int, raw r) { c += Lg::key(r) == border; });
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane < C) put(remote(&s_cnt[seg_id], lane), c);
    sync();
    int before = 0, owner = -1, skip = 0;
    for (int i = 0; i < segs; ++i) {
      if (before < ties && ties <= before + s_cnt[i]) {
        owner = i;
        skip = ties - before;  // its skip-th tie is the last
      }
      before += s_cnt[i];
    }
    if (owner == seg_id) {
      int found = -1;
      for (int gb = g0; gb < g1 && found < 0; gb += 32) {
        const uint4 v = part[gb + lane];
        int mine = 0;
#pragma unroll
        for (int e = 0; e < GROUP; ++e) mine += Lg::key(Lg::at(v, e)) == border;
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        int at = -1, left = skip - (inc - mine);
        if (left > 0 && left <= mine) {
#pragma unroll
          for (int e = 0; e < GROUP; ++e)
            if (Lg::key(Lg::at(v, e)) == border && --left == 0) at = (gb + lane) * GROUP + e;
        }
        const uint32_t who = __ballot_sync(0xffffffffu, at >= 0);
        if (who) found = __shfl_sync(0xffffffffu, at, __ffs(who) - 1);
        skip -= __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane < C) {
        put(remote(&s_cut[0], lane), found);
        put(remote(&s_cut[1], lane), rank);
      }
    }
    sync();
    cut = (long long)s_cut[1] * n + s_cut[0];
  }
  // ---- kept weights by index, and the token ----
  auto weight_of = [&](int i, raw r) {  // of place i of this part, 0 if it is not kept
    const uint32_t key = Lg::key(r);
    const bool kept = r != NEG && (key > border || (key == border && first + i <= cut));
    return kept ? weigh(Lg::value(r)) : Sum2{0.f, 0.f};
  };
  Sum2 total{0.f, 0.f};
  if (alive) {
    Sum2 s{0.f, 0.f};
    each([&](int i, raw r) {
      const Sum2 w = weight_of(i, r);
      if (w.hi > 0.f) s = sum_of(s, w);
    });
    s = warp_sum(s);
    if (lane < C) put(remote(&s_warp[round & 1][0][seg_id], lane), s.hi, s.lo);
    sync();
    // The first of values v[0 .. count) (one or more per lane) whose cumulative sum, from
    // `base` on, exceeds `aim`; the last above 0 if none does.  *base: the sum before it.
    auto find = [&](const float2* v, int count, Sum2 aim, Sum2* base) {
      const int per = (count + 31) / 32, i0 = lane * per;
      Sum2 mine{0.f, 0.f};
      for (int i = i0; i < min(i0 + per, count); ++i) mine = sum_of(mine, Sum2{v[i].x, v[i].y});
      const Sum2 inc = warp_sums(mine);
      Sum2 c = {__shfl_up_sync(0xffffffffu, inc.hi, 1), __shfl_up_sync(0xffffffffu, inc.lo, 1)};
      c = lane ? sum_of(*base, c) : *base;
      int hit = -1, last = -1;
      Sum2 at_hit = c, at_last = c;
      for (int i = i0; i < min(i0 + per, count); ++i) {
        const Sum2 w = {v[i].x, v[i].y}, after = sum_of(c, w);
        if (w.hi > 0.f) {
          last = i;
          at_last = c;
          if (hit < 0 && exceeds(after, aim)) {
            hit = i;
            at_hit = c;
          }
        }
        c = after;
      }
      const uint32_t hits = __ballot_sync(0xffffffffu, hit >= 0);
      const uint32_t lasts = __ballot_sync(0xffffffffu, last >= 0);
      const int l = hits ? __ffs(hits) - 1 : (lasts ? 31 - __clz((int)lasts) : 0);
      *base = hits ? lane_of(at_hit, l) : lane_of(at_last, l);
      return __shfl_sync(0xffffffffu, hits ? hit : last, l);
    };
    if (warp == 0) {
      const float2* const v = s_warp[round & 1][0];
      Sum2 all{0.f, 0.f};
      for (int i = lane; i < segs; i += 32) all = sum_of(all, Sum2{v[i].x, v[i].y});
      all = warp_sum(all);
      const float u = p.u[row];
      const Sum2 aim = times(all, u > 0.f ? fminf(u, 2.f) : 0.f);
      Sum2 base{0.f, 0.f};
      const int owner = find(v, segs, aim, &base);
      if (lane == 0) {
        s_i[0] = owner;
        s_f[2] = aim.hi;
        s_f[3] = aim.lo;
        s_f[4] = base.hi;
        s_f[5] = base.lo;
        s_f[6] = all.hi;
        s_f[7] = all.lo;
      }
    }
    __syncthreads();
    total = Sum2{s_f[6], s_f[7]};
    if (s_i[0] / sa::WARPS == rank) {
      // The segment's steps of 32 groups, a warp each, then the step's elements.
      const int s0 = (s_i[0] % sa::WARPS) * (p.seg / GROUP), steps = p.seg / GROUP / 32;
      for (int st = warp; st < steps; st += sa::WARPS) {
        const int g = s0 + st * 32 + lane;
        const uint4 v = part[g];
        Sum2 mine{0.f, 0.f};
#pragma unroll
        for (int e = 0; e < GROUP; ++e) mine = sum_of(mine, weight_of(g * GROUP + e, Lg::at(v, e)));
        mine = warp_sum(mine);
        if (lane == 0) s_steps[st] = make_float2(mine.hi, mine.lo);
      }
      __syncthreads();
      if (warp == 0) {
        const Sum2 aim = {s_f[2], s_f[3]};
        Sum2 base = {s_f[4], s_f[5]};
        const int st = find(s_steps, steps, aim, &base);
        const int g = s0 + st * 32 + lane;
        const uint4 v = part[g];
        Sum2 w[GROUP], mine{0.f, 0.f};
#pragma unroll
        for (int e = 0; e < GROUP; ++e) {
          w[e] = weight_of(g * GROUP + e, Lg::at(v, e));
          mine = sum_of(mine, w[e]);
        }
        const Sum2 inc = warp_sums(mine);
        Sum2 c = {__shfl_up_sync(0xffffffffu, inc.hi, 1), __shfl_up_sync(0xffffffffu, inc.lo, 1)};
        c = lane ? sum_of(base, c) : base;
        int hit = -1, last = -1;
#pragma unroll
        for (int e = 0; e < GROUP; ++e) {
          c = sum_of(c, w[e]);
          if (w[e].hi > 0.f) {
            last = g * GROUP + e;
            if (hit < 0 && exceeds(c, aim)) hit = last;
          }
        }
        const uint32_t hits = __ballot_sync(0xffffffffu, hit >= 0);
        const uint32_t lasts = __ballot_sync(0xffffffffu, last >= 0);
        const int l = hits ? __ffs(hits) - 1 : 31 - __clz((int)lasts);
        if (lane == l) p.tokens[row] = (int)(first + (hits ? hit : last) - lead);
      }
    }
  } else if (rank == 0 && t == 0) {
    p.tokens[row] = -1;
  }
  if (p.probs) {
    // 1 / total as two floats.
    const float i_hi = alive ? __frcp_rn(total.hi) : 0.f;
    const float i_lo = -i_hi * __fmaf_rn(total.lo, i_hi, __fmaf_rn(total.hi, i_hi, -1.f));
    float* const dst = p.probs + row * p.V;
    const raw* const mine = reinterpret_cast<const raw*>(smem_raw);
    for (int i = t; i < n; i += sa::THREADS) {
      const long long e = first + i - lead;
      if (e < 0 || e >= p.V) continue;
      float q = 0.f;
      if (alive) {
        const Sum2 w = weight_of(i, mine[i]);
        q = __fmaf_rn(w.hi, i_hi, __fmaf_rn(w.hi, i_lo, __fmul_rn(w.lo, i_hi)));
      }
      dst[e] = q;
    }
  }
  // No CTA leaves while another may still read its bins or write its sums.
  if (C > 1) sync();
}

template <typename T>
static cudaError_t launch_sample(SampleParams& p, long long rows, cudaStream_t stream) {
  static int attr_set[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE)) {
    e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             sa::SMEM_MAX);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) __atomic_store_n(&attr_set[dev], 1, __ATOMIC_RELEASE);
  }
  const size_t smem = (size_t)p.seg * sa::WARPS * sizeof(T);
  return launch_dependent(sample_kernel<T>, dim3((unsigned)(rows * p.cluster)), sa::THREADS, stream,
                          p, p.cluster, smem);
}

}  // namespace fa

static bool al(const void* p, unsigned n) {
  return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

extern "C" int fa_sample(const void* logits, const float* uniforms, const float* temperature,
                         const int32_t* top_k, const float* top_p, const float* min_p,
                         int32_t* tokens, float* probs, int rows, int V, long long row_stride,
                         int dtype, cudaStream_t stream) {
  if (rows < 0 || V < 1 || row_stride < V) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP16 && dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (rows > INT32_MAX / fa::sa::CLUSTER) return FA_ERR_INVALID_ARG;
  const int es = dtype == FA_FP32 ? 4 : 2, group = 16 / es;
  // A part per CTA: whole steps of 32 groups for each warp.
  const int step = 32 * group;
  auto seg_of = [&](int cluster) {
    const long long segs = (long long)cluster * fa::sa::WARPS;
    return ((V + group - 1 + segs - 1) / segs + step - 1) / step * step;
  };
  if (seg_of(fa::sa::CLUSTER) * fa::sa::WARPS * es > fa::sa::SMEM_MAX) return FA_ERR_UNSUPPORTED;
  if (rows == 0) return FA_OK;
  if (!al(logits, es) || !al(uniforms, 4) || !al(tokens, 4)) return FA_ERR_INVALID_ARG;
  if ((temperature && !al(temperature, 4)) || (top_k && !al(top_k, 4)) ||
      (top_p && !al(top_p, 4)) || (min_p && !al(min_p, 4)) || (probs && !al(probs, 4)))
    return FA_ERR_INVALID_ARG;
  const fa::SetupDuringCapture setup;
  fa::SampleParams p = {};
  p.logits = logits;
  p.u = uniforms;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.tokens = tokens;
  p.probs = probs;
  p.stride = row_stride;
  p.V = V;
  const int sms = fa::sm_count() > 0 ? fa::sm_count() : 148;
  p.cluster = fa::sa::CLUSTER;
  while (p.cluster > 1 && seg_of(p.cluster / 2) * fa::sa::WARPS * es <= fa::sa::SMEM_MAX &&
         ((long long)rows * p.cluster > 2ll * sms || seg_of(p.cluster / 2) <= 2 * step))
    p.cluster /= 2;
  p.seg = (int)seg_of(p.cluster);
  cudaError_t e;
  if (dtype == FA_FP32)
    e = fa::launch_sample<float>(p, rows, stream);
  else if (dtype == FA_BF16)
    e = fa::launch_sample<__nv_bfloat16>(p, rows, stream);
  else
    e = fa::launch_sample<__half>(p, rows, stream);
  return fa::record_cuda_status(e, "sampling launch");
}
