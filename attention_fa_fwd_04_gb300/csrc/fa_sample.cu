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
// No row is sorted.  The border is found by narrowing an interval of keys (the
// logits' bits, made to order as whole numbers).
//   top-k   The k-th largest of the threads' largest logits is a lower bound of the k-th
//           logit, and for k up to a third of the threads few more than k lie above it:
//           those become a list that every CTA ranks, and draws from.  Larger k (and rows
//           of many equal logits): passes that count the interval's keys in 2048 bins.
//   top-p   One pass counts logits in bins of 1/64 of the temperature, which says within
//           about a bin where the border is; the next adds up exactly everything and what
//           is above those bins, and lists what is in them (or counts it, where that is
//           much); the list's weights then give the border.  Whatever the estimate
//           missed, the sums show, and the search goes on from there; after ten rounds it
//           halves, so that 42 are the most that any row takes (8 rows of 5000 nearly equal
//           logits with top_p = 1 - 2^-20, 22 rounds: 113 us; where the estimate holds, 14).
//
// The answers are whole numbers.  With 128000 tokens an error of 1e-7 in the sums
// would move one draw in fifty, so weights are pairs of floats good to 2^-31 (most to
// 2^-33; sums to 2^-36), added as pairs in a fixed order.  A weight and its addition take
// 8 clocks of an SM for 64 tokens (packed fp32 arithmetic; the table has a copy for every
// second lane: one of 1024 entries without copies took 16, its reads met in the banks;
// fp64 would be bound by the few fp64 units).
//
// Layout: a cluster of up to 8 CTAs takes a row and keeps it in shared memory, so
// that HBM is read once however many passes there are.  Every thread has consecutive
// tokens, so that its sums are also what finds the token in the end.
//
// Measured (device time of one call in a captured sequence): 10.7 us for one row of 32000
// fp32 logits with top-k of 50 and top-p (15.1 with top-k of 300, 16 to 18 with top-p alone),
// 43.6 for 64 rows of 128000 bf16 with top-p and min-p (HBM's share is 2.4), 26.8 for 200 of
// 50257 fp16 with temperature alone (3.0), 97 to 99 for 512 of 32000 fp32 with top-k, top-p and
// the distributions written (19.4).  64 registers hold two CTAs per SM; the compiler spills 196
// bytes of stores there (fp32; 244 for the 16-bit types).  What bounds it: the two passes of
// weights (about half of a row's time with top-p), and the chain of meetings, scans and
// rankings between them (some 20000 clocks), of which two resident CTAs hide part.
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
constexpr int LIST = 512;              // tokens that a CTA ranks
constexpr int SMEM_MAX = 176 * 1024;   // bytes of a CTA's part of a row
constexpr int TRIES = 10;              // rounds of top-p's search before it halves
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
  int groups;  // 16-byte groups of the row per thread
};

// Logits as they are stored, and their order as whole numbers, their keys (NaN counts as
// -infinity, -0 as 0).  Negative numbers' keys are their distance below 0's, so that -0 has
// none of its own: neighbouring keys are different values, and a comparison of values is one
// of keys.  (The search relies on that: a key past its bounds would be past the bins.)
template <typename T>
struct Logits;
template <>
struct Logits<float> {
  typedef uint32_t raw;
  static constexpr int GROUP = 4;  // elements of 16 bytes
  static __device__ __forceinline__ float2 pair(const uint4& g, int x) {
    return x == 0 ? make_float2(__uint_as_float(g.x), __uint_as_float(g.y))
                  : make_float2(__uint_as_float(g.z), __uint_as_float(g.w));
  }
  static constexpr raw NEG = 0xff800000u;
  static __device__ __forceinline__ float value(raw r) { return __uint_as_float(r); }
  static __device__ __forceinline__ raw clean(raw r) {
    const float x = __uint_as_float(r);
    return __float_as_uint(fmaxf(x + 0.f, -INFINITY));  // (of a NaN and a number, the number)
  }
  static __device__ __forceinline__ uint32_t key(raw r) {
    return r & 0x80000000u ? 0u - r : r | 0x80000000u;
  }
  static __device__ __forceinline__ raw unkey(uint32_t k) {
    return k & 0x80000000u ? k ^ 0x80000000u : 0u - k;
  }
  static __device__ __forceinline__ float clean(uint4& g) {  // all of a group's; the largest
    g = make_uint4(clean(g.x), clean(g.y), clean(g.z), clean(g.w));
    return fmaxf(fmaxf(__uint_as_float(g.x), __uint_as_float(g.y)),
                 fmaxf(__uint_as_float(g.z), __uint_as_float(g.w)));
  }
  // (Rounds up where the type is narrower.)
  static __device__ __forceinline__ raw from(float x) { return clean(__float_as_uint(x)); }
};
__device__ __forceinline__ uint32_t word(const uint4& g, int x) {
  return x == 0 ? g.x : x == 1 ? g.y : x == 2 ? g.z : g.w;
}
template <typename H>
struct Logits16 {
  typedef uint16_t raw;
  static constexpr int GROUP = 8;
  static __device__ __forceinline__ uint32_t key(raw r) {
    return r & 0x8000u ? (uint16_t)(0u - r) : (uint16_t)(r | 0x8000u);
  }
  static __device__ __forceinline__ raw unkey(uint32_t k) {
    return k & 0x8000u ? (raw)(k ^ 0x8000u) : (raw)(0u - k);
  }
};
template <>
struct Logits<__nv_bfloat16> : Logits16<__nv_bfloat16> {
  static constexpr raw NEG = 0xff80u;
  static __device__ __forceinline__ float value(raw r) { return __uint_as_float((uint32_t)r << 16); }
  static __device__ __forceinline__ float2 pair(const uint4& g, int x) {
    const uint32_t w = word(g, x);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ raw clean(raw r) {
    return (r & 0x7fffu) > 0x7f80u ? NEG : (r == 0x8000u ? (raw)0 : r);
  }
  static __device__ __forceinline__ float clean(uint4& g) {  // all of a group's; the largest
    const __nv_bfloat162 neg = __bfloat162bfloat162(__ushort_as_bfloat16(NEG));
    const __nv_bfloat162 zero = __bfloat162bfloat162(__ushort_as_bfloat16(0));
    __nv_bfloat162* const x = reinterpret_cast<__nv_bfloat162*>(&g);
    __nv_bfloat162 m = neg;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __hmax2(__hadd2(x[i], zero), neg);  // (of a NaN and a number, the number)
      m = __hmax2(m, x[i]);
    }
    return fmaxf(__bfloat162float(m.x), __bfloat162float(m.y));
  }
  static __device__ __forceinline__ raw from(float x) {
    return clean(__bfloat16_as_ushort(__float2bfloat16_ru(x)));
  }
};
template <>
struct Logits<__half> : Logits16<__half> {
  static constexpr raw NEG = 0xfc00u;
  static __device__ __forceinline__ float value(raw r) { return __half2float(__ushort_as_half(r)); }
  static __device__ __forceinline__ float2 pair(const uint4& g, int x) {
    const uint32_t w = word(g, x);
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ raw clean(raw r) {
    return (r & 0x7fffu) > 0x7c00u ? NEG : (r == 0x8000u ? (raw)0 : r);
  }
  static __device__ __forceinline__ float clean(uint4& g) {  // all of a group's; the largest
    const __half2 neg = __half2half2(__ushort_as_half(NEG));
    const __half2 zero = __half2half2(__ushort_as_half(0));
    __half2* const x = reinterpret_cast<__half2*>(&g);
    __half2 m = neg;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = __hmax2(__hadd2(x[i], zero), neg);  // (of a NaN and a number, the number)
      m = __hmax2(m, x[i]);
    }
    return fmaxf(__half2float(m.x), __half2float(m.y));
  }
  static __device__ __forceinline__ raw from(float x) {
    return clean(__half_as_ushort(__float2half_ru(x)));
  }
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
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) a = sum_of(a, shfl_xor(a, o));
  return a;
}
__device__ __forceinline__ void warp_sum(Sum2& a, Sum2& b) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    a = sum_of(a, shfl_xor(a, o));
    b = sum_of(b, shfl_xor(b, o));
  }
}
// Sums of the lanes up to this one.
__device__ __forceinline__ Sum2 warp_sums(Sum2 a) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const Sum2 y = {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
    if (lane >= o) a = sum_of(y, a);
  }
  return a;
}
__device__ __forceinline__ Sum2 lane_of(Sum2 a, int l) {
  return {__shfl_sync(0xffffffffu, a.hi, l), __shfl_sync(0xffffffffu, a.lo, l)};
}

__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }
// Sums of weights hi + hi q, two at once.  The sums begin at 2, the largest weight, so
// that a sum's rounding is what three operations give.
struct Sums {
  float2 hi = {2.f, 2.f}, lo = {0.f, 0.f};
  __device__ __forceinline__ void add(float2 h, float2 q) {
    const float2 s = __fadd2_rn(hi, h), t = __fadd2_rn(s, make_float2(-hi.x, -hi.y));
    lo = __fadd2_rn(__ffma2_rn(h, q, lo), __fadd2_rn(h, make_float2(-t.x, -t.y)));
    hi = s;
  }
  __device__ __forceinline__ Sum2 all() const {
    return sum_of(sum_of(hi.x - 2.f, lo.x), sum_of(hi.y - 2.f, lo.y));
  }
};

// Weights of a row's logits, up to a power of two that all of them share.  In y =
// (l - base) log2(e) / T = k / 128 + a, |a| <= 2^-8, 2^y = 2^(k / 128) 2^a: a table has the
// first factor, a polynomial the second.  With base = 0, l needs no exact difference;
// where |top| / T is so large that y would lose bits, base = top, and the differences that
// matter (l within T of top) are exact.
struct Weigher {
  float shift;            // -base
  float s_hi, s_lo;       // log2(e) / T
  float lowest;           // l - base that has no weight any more: 2^-126 of the largest
  float magic;            // 1.5 * 2^16, which rounds to 1 / 128, and the exponents' bias
  const float2* table;    // this lane's copy: entries 16 apart, no two lanes in one bank
  // Weights of v: hi + hi * q, |q| < 2^-8.
  __device__ __forceinline__ void operator()(float2 v, float2* hi, float2* q) const {
    float2 d = __fadd2_rn(v, twice(shift));
    d = make_float2(fmaxf(d.x, lowest), fmaxf(d.y, lowest));
    const float2 t = __ffma2_rn(d, twice(s_hi), twice(magic));
    const float2 r = __ffma2_rn(d, twice(s_hi), __fadd2_rn(twice(magic), make_float2(-t.x, -t.y)));
    const float2 a = __ffma2_rn(d, twice(s_lo), r);
    // ln 2, (ln 2)^2 / 2, (ln 2)^3 / 6.
    float2 f = __ffma2_rn(a, twice(0.0555041086648215800f), twice(0.240226506959100712f));
    f = __ffma2_rn(a, f, twice(0.693147180559945309f));
    const uint32_t bx = __float_as_uint(t.x), by = __float_as_uint(t.y);
    const float2 tx = table[(bx & 127u) * 16], ty = table[(by & 127u) * 16];
    // t's bits from the seventh on are the factor's exponent; 0 where l is `lowest`.
    const float2 e = make_float2(__uint_as_float((bx << 16) & 0xff800000u),
                                 __uint_as_float((by << 16) & 0xff800000u));
    *hi = __fmul2_rn(make_float2(tx.x, ty.x), e);
    *q = __ffma2_rn(a, f, make_float2(tx.y, ty.y));
  }
  __device__ __forceinline__ Sum2 one(float v) const {
    float2 h, q;
    (*this)(twice(v), &h, &q);
    return {h.x, __fmul_rn(h.x, q.x)};
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
__device__ __forceinline__ int add_remote(uint32_t at, int a) {
  int r;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(at), "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ int get(uint32_t at) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
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
__global__ void __launch_bounds__(sa::THREADS, 2) sample_kernel(const __grid_constant__ SampleParams p) {
  using Lg = Logits<T>;
  using raw = typename Lg::raw;
  constexpr raw NEG = Lg::NEG;
  constexpr int GROUP = Lg::GROUP;
  constexpr int AHEAD = 8;
  constexpr uint32_t NEGS = sizeof(raw) == 2 ? NEG * 0x10001u : NEG;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  __shared__ float2 s_table[128 * 16];
  __shared__ __align__(16) uint32_t s_hist[2][sa::BINS];
  __shared__ float2 s_first[sa::SEGS];       // every warp's largest logit, smallest lane maximum
  __shared__ float2 s_warp[2][2][sa::SEGS];  // per round and quantity: every warp's sum
  __shared__ int s_cnt[sa::SEGS];
  // Tokens to rank: key, index inverted.  Every CTA of the cluster writes every CTA's list, so
  // between the reading of one and the writing of the next there is a cluster barrier: of a
  // round in between, or its own (at the end of top-p's loop).
  __shared__ __align__(16) unsigned long long s_list[sa::LIST + 8];
  __shared__ int s_rank[sa::LIST];
  __shared__ float2 s_block[sa::WARPS + 1];
  __shared__ uint32_t s_scan[sa::WARPS];
  __shared__ float s_fscan[sa::WARPS];
  __shared__ int s_i[4], s_cut, s_listed[4];
  __shared__ uint32_t s_border;
  __shared__ float2 s_pair[5];
  constexpr uint32_t NONE = 0xffffffffu;
  // A bin (11 bits), how many of its key (20), whether that is fewer than it has (where a bin
  // is more than a key: whether few lie in it).
  __shared__ uint32_t s_found;
  __shared__ float2 s_low;  // T ln(min_p)
  __shared__ float s_from;  // a bound of the lanes' maxima that matter
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int C = p.cluster;
  const int rank = (int)(blockIdx.x & (unsigned)(C - 1));  // (C is 1, 2, 4 or 8)
  const long long row = blockIdx.x >> (__ffs(C) - 1);
  const int segs = C * sa::WARPS, seg_id = rank * sa::WARPS + warp;
  const int own = p.groups;  // 16-byte groups per thread, consecutive in the row
  const int n = own * GROUP * sa::THREADS;  // elements of this CTA's part
  pdl_launch_dependents();
  for (int i = t; i < 128 * 16; i += sa::THREADS)
    s_table[i] = make_float2(kExp2Table[i >> 4][0], kExp2Table[i >> 4][1]);
  for (int i = t; i < 2 * sa::BINS; i += sa::THREADS) (&s_hist[0][0])[i] = 0;
  s_rank[t] = 0;
  if (t < 8) s_list[sa::LIST + t] = 0;
  static_assert(sa::LIST == sa::THREADS, "an item of the list per thread");
  if (t < 4) s_listed[t] = 0;
  pdl_wait_primary();

  auto arrive = [] { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); };
  auto wait = [] { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); };
  auto sync = [&] {  // the cluster's CTAs meet; what they stored is visible
    if (C > 1) {
      arrive();
      wait();
    } else {
      __syncthreads();
    }
  };
  if (C > 1) arrive();  // (waited for below: no CTA is written to before it runs)
  // ---- the row into shared memory, its largest logit ----
  const T* const src = static_cast<const T*>(p.logits) + row * p.stride;
  const int lead = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  const int first = rank * n - lead;  // token of this part's first element
  uint4* const part = reinterpret_cast<uint4*>(smem_raw);
  float temp = p.temperature ? p.temperature[row] : 1.f;
  const bool greedy = !(temp > 0.f);
  // (Once, for the weights, min-p's border and the search's steps alike.)
  temp = greedy ? 1.f : fminf(fmaxf(temp, 0x1p-99f), 0x1p99f);
  const int k = p.top_k ? p.top_k[row] : 0;
  const float tp = p.top_p ? p.top_p[row] : 1.f;
  const float mp = p.min_p ? p.min_p[row] : 0.f;
  const float u = p.u[row];
  const float uu = u > 0.f ? fminf(u, 2.f) : 0.f;
  float mx = -INFINITY;
  {
    const int g0 = warp * 32 * own, from = first + g0 * GROUP;  // this warp's
    // Eight loads ahead of what is done with them.
    const uint4* const at = reinterpret_cast<const uint4*>(src + from);
    for (int i0 = lane; i0 < 32 * own; i0 += 32 * AHEAD) {
      uint4 v[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int i = i0 + 32 * j, e = from + i * GROUP;
        v[j] = make_uint4(NEGS, NEGS, NEGS, NEGS);
        if (i < 32 * own && e >= 0 && e + GROUP <= p.V) v[j] = at[i];
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const int i = i0 + 32 * j, e = from + i * GROUP;
        if (i >= 32 * own) break;
        if ((e < 0 && e + GROUP > 0) || (e < p.V && e + GROUP > p.V)) {  // the row's ends
          alignas(16) raw x[GROUP];
#pragma unroll
          for (int y = 0; y < GROUP; ++y)
            x[y] = e + y >= 0 && e + y < p.V ? reinterpret_cast<const raw*>(src)[e + y] : NEG;
          v[j] = *reinterpret_cast<uint4*>(x);
        }
        mx = fmaxf(mx, Lg::clean(v[j]));
        part[g0 + i] = v[j];
      }
    }
  }
  if (t == sa::THREADS - 32 && mp > 0.f) {
    const double x = fmin((double)temp * log((double)mp), 0.0);  // (above 1: one token is kept)
    s_low = make_float2((float)x, (float)(x - (double)(float)x));
  }
  {
    float hi = mx, lo = mx;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    }
    if (C > 1) wait();
    if (lane < C) put(remote(&s_first[seg_id], lane), hi, lo);
  }
  // log2(e) / T in two floats.
  Weigher weigh;
  weigh.table = s_table + (lane & 15);
  {
    const float inv = __fdividef(1.f, temp);  // (what it is off by goes into s_lo)
    weigh.s_hi = 1.44269502162933349609f * inv;
    weigh.s_lo = __fmul_rn(inv, __fadd_rn(__fmaf_rn(-weigh.s_hi, temp, 1.44269502162933349609f),
                                          1.92596299112661746887e-8f));
  }
  sync();
  float top = -INFINITY;
  for (int i = lane; i < segs; i += 32) top = fmaxf(top, s_first[i].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));

  // Every group of this thread's: f(its index in the part, the group).  The lanes begin
  // at different ones, so that they read different banks.
  const int even = own % 8 == 0 ? 8 : own % 4 == 0 ? 4 : own % 2 == 0 ? 2 : 1;
  const int begin = (lane & 7) * even >> 3;
  auto each = [&](auto&& f) {
    int x = begin;
#pragma unroll 1
    for (int g = 0; g < own; ++g) {
      const int i = t * own + x;
      f(i, part[i]);
      if (++x == own) x = 0;
    }
  };
  // Which elements of a group lie in [lo, hi], as bits; f(raw value, index in the part) of
  // those (few: the loop is as long as the fullest lane's).
  auto within = [](uint4 g, float lo, float hi) {
    uint32_t m = 0;
#pragma unroll
    for (int x = 0; x < GROUP / 2; ++x) {
      const float2 v = Lg::pair(g, x);
      if (v.x >= lo && v.x <= hi) m |= 1u << (2 * x);
      if (v.y >= lo && v.y <= hi) m |= 2u << (2 * x);
    }
    return m;
  };
  auto each_of = [&](uint32_t m, int i, auto&& f) {
#pragma unroll 1
    for (; m; m &= m - 1) {
      const int x = i * GROUP + __ffs((int)m) - 1;
      f(reinterpret_cast<const raw*>(part)[x], x);
    }
  };
  // Logits of +infinity share the weight: they become 0 and all others -infinity.
  const bool was_inf = top == INFINITY;
  if (was_inf) {
    mx = -INFINITY;
    each([&](int i, uint4 g) {
      alignas(16) raw x[GROUP];
      *reinterpret_cast<uint4*>(x) = g;
#pragma unroll
      for (int j = 0; j < GROUP; ++j) {
        x[j] = Lg::value(x[j]) == INFINITY ? (raw)0 : NEG;
        mx = fmaxf(mx, Lg::value(x[j]));
      }
      part[i] = *reinterpret_cast<uint4*>(x);
    });
    top = 0.f;
  }
  const bool alive = top != -INFINITY;
  const uint32_t kneg = Lg::key(NEG), kmax = Lg::key(Lg::from(top));
  {
    float y = top * weigh.s_hi;
    weigh.shift = 0.f;
    if (!(fabsf(y) < 1000.f)) {
      y = 0.f;
      weigh.shift = -top;
    }
    const float e = floorf(y);
    weigh.lowest = (e - 126.5f) / weigh.s_hi;
    weigh.magic = 98304.f + (127.f - e);
  }
  auto value_of = [&](uint32_t key) { return Lg::value(Lg::unkey(key)); };

  // Exchanges alternate between two buffers of bins and sums, so that one barrier
  // each does: a CTA fills a buffer again only after the barrier that the others
  // reach when they have read it.
  int round = 0;
  static_assert(sa::BINS == 4 * sa::THREADS, "four bins per thread");
  auto gather = [&](uint32_t (&h)[4]) {  // four bins of all CTAs together
    uint4 s = *reinterpret_cast<const uint4*>(&s_hist[round & 1][4 * t]);
    if (C > 1) {
      uint4 v[sa::CLUSTER - 1];
#pragma unroll
      for (int c = 1; c < sa::CLUSTER; ++c)
        if (c < C) v[c - 1] = get4(remote(&s_hist[round & 1][4 * t], (rank + c) & (C - 1)));
#pragma unroll
      for (int c = 1; c < sa::CLUSTER; ++c) {
        if (c < C) {
          s.x += v[c - 1].x;
          s.y += v[c - 1].y;
          s.z += v[c - 1].z;
          s.w += v[c - 1].w;
        }
      }
    }
    h[0] = s.x;
    h[1] = s.y;
    h[2] = s.z;
    h[3] = s.w;
  };
  auto turn = [&] {  // (after the barrier, and before the block's next one, which has to follow)
    *reinterpret_cast<uint4*>(&s_hist[(round & 1) ^ 1][4 * t]) = make_uint4(0, 0, 0, 0);
    // (Other CTAs add to the next round's: the one after it.)
    if (t == 0) s_listed[(round + 2) & 3] = 0;
    ++round;
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
#pragma unroll
    for (int i = 0; i < sa::WARPS; ++i) x += i < warp ? sums[i] : 0;
    return x;
  };
  // The same of pairs (in warps without any it is not computed); *all: the sum of all.
  // What every warp would compute alike one warp computes: 32 warps' instructions cost
  // more than the barrier.
  auto pairs_before = [&](Sum2 mine, Sum2* all) {
    Sum2 inc{0.f, 0.f};
    if (__any_sync(0xffffffffu, mine.hi > 0.f)) inc = warp_sums(mine);
    if (lane == 31) s_block[warp] = make_float2(inc.hi, inc.lo);
    __syncthreads();
    if (warp == 0) {
      Sum2 c = lane < sa::WARPS ? Sum2{s_block[lane].x, s_block[lane].y} : Sum2{0.f, 0.f};
      c = warp_sums(c);
      const Sum2 e = {__shfl_up_sync(0xffffffffu, c.hi, 1), __shfl_up_sync(0xffffffffu, c.lo, 1)};
      __syncwarp();
      if (lane <= sa::WARPS) s_block[lane] = lane ? make_float2(e.hi, e.lo) : make_float2(0.f, 0.f);
    }
    __syncthreads();
    *all = Sum2{s_block[sa::WARPS].x, s_block[sa::WARPS].y};
    const Sum2 c = {s_block[warp].x, s_block[warp].y};
    const Sum2 e = {__shfl_up_sync(0xffffffffu, inc.hi, 1), __shfl_up_sync(0xffffffffu, inc.lo, 1)};
    return lane ? sum_of(c, e) : c;
  };
  // The list's `count` items, mine(t) each, in falling order, in threads too; a thread
  // compares an item to a share of the others.
  auto ranked = [&](int count, unsigned long long mine) {
    const int bits = max(5, 32 - __clz(max(count - 1, 0)));
    const int item = t & ((1 << bits) - 1), parts = sa::THREADS >> bits;
    const int per = ((count + parts - 1) / parts + 7) & ~7, j0 = (t >> bits) * per;
    s_list[t] = mine;  // (0 past the last)
    __syncthreads();
    if (item < count) {
      const unsigned long long x = s_list[item];
      int before = 0;
#pragma unroll 1
      for (int j = j0; j < min(j0 + per, count); j += 8) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(s_list + j + i);
          before += (o.x > x) + (o.y > x);
        }
      }
      if (before) atomicAdd(&s_rank[item], before);
    }
    __syncthreads();
    if (t < count) {
      s_list[s_rank[t]] = mine;
      s_rank[t] = 0;
    }
    __syncthreads();
    return t < count ? s_list[t] : 0ull;
  };
  // One more for every CTA's list.
  auto enlist = [&](raw l, int x) {
    const int at = add_remote(remote(&s_listed[round & 3], 0), 1);
    if (at < sa::LIST) {
#pragma unroll 1
      for (int r = 0; r < C; ++r)
        put(remote(&s_list[at], r), __uint_as_float(~(uint32_t)(first + x)),
            __uint_as_float(Lg::key(l)));
    }
  };
  auto shift_of = [](uint32_t lo, uint32_t hi) { return max(0, 21 - __clz((int)(hi - lo))); };
  // Lane sums v from `base` on: the first lane at which they exceed `aim`, or the last
  // with any; *base: the sum before it.
  auto find = [&](Sum2 v, Sum2 aim, Sum2* base) {
    const Sum2 inc = warp_sums(v);
    Sum2 c = {__shfl_up_sync(0xffffffffu, inc.hi, 1), __shfl_up_sync(0xffffffffu, inc.lo, 1)};
    c = lane ? sum_of(*base, c) : *base;
    const bool some = v.hi > 0.f;
    const uint32_t hits = __ballot_sync(0xffffffffu, some && exceeds(sum_of(c, v), aim));
    const uint32_t lasts = __ballot_sync(0xffffffffu, some);
    const int l = hits ? __ffs(hits) - 1 : (lasts ? 31 - __clz((int)lasts) : 0);
    *base = lane_of(c, l);
    return l;
  };
  // Tokens that share a key: how many lie before this lane's segment(s) and lanes.
  auto count_before = [&](int mine) {
    int x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x - mine;
  };

  // The key below which min_p leaves nothing: w >= min_p is l >= top + T ln(min_p).
  auto lowest_key = [&] {
    if (!(mp > 0.f)) return kneg;
    const Sum2 x = sum_of(Sum2{top, 0.f}, Sum2{s_low.x, s_low.y});
    const raw r = Lg::from(x.hi);  // (rounded up)
    return min(kmax, Lg::key(r) + (Lg::value(r) == x.hi && x.lo > 0.f ? 1u : 0u));
  };
  // What is kept: keys above `border`, and the first `ties` (by index) of those at it.
  uint32_t border = kneg;
  int ties = INT_MAX;
  bool limited = false;  // whether `ties` leaves any out
  bool done = !alive;    // the token has been written
  int cut = INT_MAX;     // the token of the last tie that is kept, where that is known
  Sum2 total{0.f, 0.f}, mine{0.f, 0.f};
  // mine: this thread's tokens of keys above `summed`, where that is not 0.
  uint32_t summed = 0;
  // This thread's tokens with the border's key.
  auto count_ties = [&] {
    int c = 0;
    const float at = value_of(border);
    each([&](int, uint4 g) {
#pragma unroll
      for (int x = 0; x < GROUP / 2; ++x) {
        const float2 v = Lg::pair(g, x);
        c += (v.x == at) + (v.y == at);
      }
    });
    return c;
  };
  // The token of the last tie that is kept (c: this thread's ties; s_cnt has the warps').
  auto find_cut = [&](int c) {
    int in[4], sum = 0;
    const int per = (segs + 31) / 32;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      in[i] = i < per && lane * per + i < segs ? s_cnt[lane * per + i] : 0;
      sum += in[i];
    }
    int before = count_before(sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (Before this warp's: as its lane says.)
      if (lane * per + i == seg_id && i < per) s_rank[warp] = before;
      before += in[i];
    }
    __syncwarp();
    int skip = ties - s_rank[warp] - count_before(c);  // its skip-th tie is the last
    __syncwarp();
    if (lane == 0) s_rank[warp] = 0;
    if (skip >= 1 && skip <= c) {
      const raw at = Lg::unkey(border);
      const raw* const e = reinterpret_cast<const raw*>(part) + t * own * GROUP;
      int i = 0;
#pragma unroll 1
      for (; i < own * GROUP; ++i)
        if (e[i] == at && --skip == 0) break;
      for (int r = 0; r < C; ++r) put(remote(&s_cut, r), first + t * own * GROUP + i);
    }
    sync();
    return s_cut;
  };
  if (alive && (greedy || k == 1 || tp <= 0.f || mp > 1.f)) {
    border = kmax;
    ties = 1;
    limited = true;
  } else if (alive) {
    if (k > 0 && k < p.V) {
      // The k-th largest of the lanes' maxima is no larger than the k-th largest logit,
      // and for a small k few more than k logits are above it.
      uint32_t lo = kneg + 1, hi = kmax;
      const int w = (k + 31) / 32;
      if (k <= 3 * sa::LIST / 4 && 3 * k <= sa::THREADS * C) {
        // Where the k-th of the maxima is, in 512 bins from the top down to the w-th largest of
        // the warps' smallest ones.
        if (t < segs) {
          const float least = s_first[t].y;
          int above = 0;
#pragma unroll 8
          for (int i = 0; i < segs; ++i) {
            const float o = s_first[i].y;
            above += o > least || (o == least && i < t);
          }
          if (above == w - 1) s_from = was_inf ? -INFINITY : least;
        }
        __syncthreads();
        // (A range that is too small, or too large, to divide by counts as one bin.)
        const float from = s_from, range = top - from;
        const float per = range > 0x1p-100f ? __fdividef((float)(sa::THREADS - 1), range) : 0.f;
        if (mx >= from)
          atomicAdd(&s_hist[round & 1][min((int)((top - mx) * per), sa::THREADS - 1)], 1u);
        sync();
        uint32_t h = s_hist[round & 1][t];
#pragma unroll
        for (int c = 1; c < sa::CLUSTER; ++c)
          if (c < C) h += (uint32_t)get(remote(&s_hist[round & 1][t], (rank + c) & (C - 1)));
        turn();
        const uint32_t before = sum_before(h, s_scan);
        if (before < (uint32_t)k && (uint32_t)k <= before + h) s_i[0] = t;  // the k-th's bin
        __syncthreads();
        const float bound = top - __fdividef((float)s_i[0] + 1.01f, per);
        lo = range == 0.f ? kmax : max(lo, Lg::key(Lg::from(bound)));
        const float least_listed = value_of(lo);
        each([&](int i, uint4 g) {
          each_of(within(g, least_listed, INFINITY), i, enlist);
        });
        sync();
        const int have = get(remote(&s_listed[round & 3], 0));
        turn();
        if (have <= sa::LIST) {
          // (All CTAs alike.)
          int count = have;
          unsigned long long x = t < have ? s_list[t] : 0;
          Sum2 all;
#pragma unroll 1
          for (int by_index = 0; by_index < 2; ++by_index) {
            // The list in order: by logit, then what is kept of it by index.
            x = ranked(count, x);
            const uint32_t key = (uint32_t)(by_index ? x : x >> 32);
            const uint32_t place = ~(uint32_t)(by_index ? x >> 32 : x);
            bool keep = t < (by_index ? count : min(have, k));
            Sum2 w{0.f, 0.f};
            if (keep) w = weigh.one(value_of(key));
            const Sum2 before = pairs_before(w, &all);
            if (!by_index) {
              if (tp < 1.f) keep = keep && (t == 0 || exceeds(times(all, tp), before));
              keep = keep && (t == 0 || key >= lowest_key());
              count = __syncthreads_count(keep);
              if (t == count - 1) {
                s_border = key;
                s_i[3] = (int)place;
                s_i[0] = INT_MAX;
                s_i[1] = -1;
              }
              x = t < count ? x << 32 | x >> 32 : 0;
            } else {
              // The first that exceeds the aim, or the last with any weight.
              const bool some = w.hi > 0.f;
              if (some && exceeds(sum_of(before, w), times(all, uu))) atomicMin(&s_i[0], t);
              if (some) atomicMax(&s_i[1], t);
              __syncthreads();
              if (rank == 0 && t == (s_i[0] < INT_MAX ? s_i[0] : s_i[1])) p.tokens[row] = (int)place;
            }
          }
          done = true;
          total = all;
          cut = s_i[3];
          border = s_border;
        } else {
          __syncthreads();  // (the bins are zero before anybody counts in them)
        }
      }
      // The border by counts: 2048 bins per pass.  (With fewer than k finite logits all stay.)
      int above = 0;
      while (!done) {
        const int shift = shift_of(lo, hi);
        const uint32_t span = hi - lo;
        uint32_t* const hist = s_hist[round & 1];
        if (t == 0) s_i[0] = -1;
        each([&](int i, uint4 g) {
#pragma unroll
          for (int x = 0; x < GROUP; ++x) {
            const uint32_t d = hi - Lg::key(reinterpret_cast<const raw*>(&g)[x]);
            if (d <= span) atomicAdd(&hist[d >> shift], 1u);
          }
        });
        sync();
        uint32_t h[4];
        gather(h);
        turn();
        uint32_t before = (uint32_t)above + sum_before(h[0] + h[1] + h[2] + h[3], s_scan);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (before < (uint32_t)k && (uint32_t)k <= before + h[e]) {
            s_i[0] = 4 * t + e;
            s_i[1] = (int)before;
            s_i[2] = (int)h[e];
          }
          before += h[e];
        }
        __syncthreads();
        const int b = s_i[0], in = s_i[2];
        if (b < 0) break;
        above = s_i[1];
        const uint32_t new_hi = hi - ((uint32_t)b << shift), width = (1u << shift) - 1;
        lo = new_hi - lo > width ? new_hi - width : lo;
        hi = new_hi;
        if (lo == hi) {
          border = hi;
          ties = k - above;
          limited = in > ties;
          break;
        }
        __syncthreads();
      }
    }
    const uint32_t lowest = lowest_key();
    if (!done && tp < 1.f) {
      if (border > kneg) {
        // What top-k leaves out goes.
        if (limited) {
          const int c = count_ties(), in_warp = __reduce_add_sync(0xffffffffu, c);
          if (lane < C) put(remote(&s_cnt[seg_id], lane), in_warp);
          sync();
          cut = find_cut(c);
        }
        each([&](int i, uint4) {
          raw* const e = reinterpret_cast<raw*>(part + i);
#pragma unroll
          for (int x = 0; x < GROUP; ++x) {
            const uint32_t key = Lg::key(e[x]);
            if (key < border || (key == border && first + i * GROUP + x > cut)) e[x] = NEG;
          }
        });
        border = kneg;
        limited = false;
        cut = INT_MAX;
      }
      // Keys in [elo, ehi] hold the border; `above` is the weight of those above.
      uint32_t elo = kneg, ehi = kmax, blo = elo, bhi = ehi;
      Sum2 above{0.f, 0.f}, target{0.f, 0.f};
      bool list = false;  // whether few keys lie in [blo, bhi], to the last estimate
      {
        // Where the border may be, from counts in 2048 bins: of 1/256 of the temperature
        // for the heavy tokens (two temperatures from the top), of 1/64 below.
        uint32_t* const hist = s_hist[round & 1];
        const float per = -0.6931471805599453f * weigh.s_hi;
        const float2 fine = twice(256.f * per), coarse = twice(64.f * per);
        // Bins of the top: 1 and 385, but for what the sums' rounding to whole numbers adds.
        // (Of logits as the weights take them, less the largest where it is many temperatures from
        // 0: the bins would lose their places beside it.)
        const float2 less = twice(weigh.shift);
        const float rest = top + weigh.shift;
        const float fine0 = 8388609.f - fine.x * rest, coarse0 = 8388993.f - coarse.x * rest;
        const float fine_top = __fmaf_rn(fine.x, rest, fine0 - 8388608.f);
        const float coarse_top = __fmaf_rn(coarse.x, rest, coarse0 - 8388608.f);
        auto below_top = [&](int b) {  // in temperatures, the middle of a bin
          return b < 513 ? ((float)b - fine_top) * (1.f / 256.f)
                         : ((float)b - coarse_top) * (1.f / 64.f);
        };
        if (t == 0) s_i[3] = -1;
        each([&](int, uint4 g) {
#pragma unroll
          for (int x = 0; x < GROUP / 2; ++x) {
            const float2 v = __fadd2_rn(Lg::pair(g, x), less);
            const float2 z = __ffma2_rn(v, fine, twice(fine0));
            const float2 y = __ffma2_rn(v, coarse, twice(coarse0));
            const uint32_t a = __float_as_uint(fminf(z.x, y.x)) - 0x4b000000u;
            const uint32_t b = __float_as_uint(fminf(z.y, y.y)) - 0x4b000000u;
            if (a < sa::BINS) atomicAdd(&hist[a], 1u);
            if (b < sa::BINS) atomicAdd(&hist[b], 1u);
          }
        });
        sync();
        uint32_t h[4];
        gather(h);
        turn();
        float m4[4], sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          m4[e] = (float)h[e] * __expf(-below_top(4 * t + e));
          sum += m4[e];
        }
        float before = sum_before(sum, s_fscan), want = 0.f;
#pragma unroll
        for (int i = 0; i < sa::WARPS; ++i) want += s_fscan[i];
        want *= tp;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // (Each thread's sums have roundings of their own, so two threads may both find it; all
          // CTAs of the cluster have to take the same.)
          if (before < want && want <= before + m4[e])
            atomicMax(&s_i[3], (4 * t + e) << 1 | (h[e] <= sa::LIST / 4 ? 1 : 0));
          before += m4[e];
        }
        __syncthreads();
        if (s_i[3] >= 0) {
          // One bin to either side; the next pass finds out whether that was enough.
          const int b = s_i[3] >> 1;
          const float d = below_top(b), w = b < 511 ? 1.5f / 256.f : 1.5f / 64.f;
          list = s_i[3] & 1;
          bhi = min(max(Lg::key(Lg::from(top - temp * (d - w))), elo), ehi);
          blo = min(max(Lg::key(Lg::from(top - temp * (d + w))), elo), bhi);
        }
      }
      // Where the bins turn out not to hold the border: how far from them it is looked for
      // next.  (With all keys up to the end, whose bins are too coarse to say where it is, such
      // a row took 25 rounds: 400 rows of 300 logits 195 us, 24 this way.)
      float reach = 0.25f * temp;
      auto key_of = [](float v) { return Lg::key(Lg::from(v)); };
      bool dense = false;
      int tries = 0;
      for (bool have_total = false;; have_total = true) {
        // After TRIES rounds [elo, ehi] is halved every time, and is exact once it is 2048 keys:
        // 32 more at the most.  (Rows are mostly done after one to four.  Bins alone may leave all
        // but a 2048th of the keys every third round: 24000 rounds at a temperature of 1e-7.)
        if (++tries > sa::TRIES) {
          blo = elo;
          bhi = elo + ((ehi - elo) >> 1);
          list = false;
        }
        // Above min_p's border only what lies there counts.
        if (bhi + 1 < lowest) bhi = blo = max(lowest - 1, elo);
        const int shift = shift_of(blo, bhi);
        const uint32_t bspan = bhi - blo;
        const bool lists = list && shift > 0, exact = lists || shift == 0;
        list = false;
        uint32_t* const hist = s_hist[round & 1];
        const float vhi = value_of(bhi), vlo = value_of(blo), vtop = value_of(ehi);
        if (t == 0) s_found = NONE;
        // Weights above the bins and (the first time) of everything; counts in them.
        Sum2 my_over{0.f, 0.f}, my_every{0.f, 0.f};
        if (!have_total) {
          Sums over, every;
          each([&](int i, uint4 g) {
            uint32_t m = 0;
#pragma unroll
            for (int x = 0; x < GROUP / 2; ++x) {
              const float2 v = Lg::pair(g, x);
              float2 hi, q;
              weigh(v, &hi, &q);
              every.add(hi, q);
              const bool a = v.x > vhi, b = v.y > vhi;
              if (!a && v.x >= vlo) m |= 1u << (2 * x);
              if (!b && v.y >= vlo) m |= 2u << (2 * x);
              over.add(make_float2(a ? hi.x : 0.f, b ? hi.y : 0.f), q);
            }
            each_of(m, i, [&](raw l, int x) {
              if (lists) {
                enlist(l, x);
              } else {
                atomicAdd(&hist[(bhi - Lg::key(l)) >> shift], 1u);
              }
            });
          });
          my_over = over.all();
          my_every = every.all();
        } else {
          each([&](int i, uint4 g) {
            each_of(within(g, vlo, vtop), i, [&](raw l, int x) {
              const uint32_t key = Lg::key(l);
              if (key > bhi) {
                my_over = sum_of(my_over, weigh.one(Lg::value(l)));
              } else if (lists) {
                enlist(l, x);
              } else {
                atomicAdd(&hist[(bhi - key) >> shift], 1u);
              }
            });
          });
        }
        const int r = round & 1;
        {
          Sum2 x = my_over, y = my_every;
          warp_sum(x, y);
          if (lane < C) {
            put(remote(&s_warp[r][0][seg_id], lane), x.hi, x.lo);
            put(remote(&s_warp[r][1][seg_id], lane), y.hi, y.lo);
          }
        }
        sync();
        uint32_t h[4] = {0, 0, 0, 0};
        int have = 0;
        if (lists) {
          have = get(remote(&s_listed[round & 3], 0));
        } else {
          gather(h);
        }
        turn();
        if (warp == 0) {  // the sums of all warps
          Sum2 x{0.f, 0.f}, y{0.f, 0.f};
#pragma unroll 1
          for (int i = lane; i < segs; i += 32) {
            const float2 v = s_warp[r][0][i], w = s_warp[r][1][i];
            x = sum_of(x, Sum2{v.x, v.y});
            y = sum_of(y, Sum2{w.x, w.y});
          }
          warp_sum(x, y);
          if (lane == 0) {
            s_pair[0] = make_float2(x.hi, x.lo);
            s_pair[1] = make_float2(y.hi, y.lo);
            s_i[0] = INT_MAX;
          }
        }
        __syncthreads();
        const Sum2 A = sum_of(above, Sum2{s_pair[0].x, s_pair[0].y});
        if (!have_total) target = times(Sum2{s_pair[1].x, s_pair[1].y}, tp);
        if (have > sa::LIST) {  // (more than the estimate: by counts, then)
          __syncthreads();
          continue;
        }
        if (!exceeds(target, A) && bhi != ehi) {  // the border lies above the bins
          const uint32_t next = key_of(vhi + reach);
          blo = elo = bhi + 1;
          bhi = min(max(next, blo), ehi);
          reach *= 16.f;
          list = true;
          __syncthreads();
          continue;
        }
        mine = sum_of(mine, my_over);
        above = A;
        ehi = bhi;
        if (bhi < lowest) {  // (bhi + 1 is lowest)
          border = lowest;
          break;
        }
        // Counts times the bins' weights (exact where a bin is one key).
        auto weight_of = [&](int e) {
          const uint32_t off = ((uint32_t)(4 * t + e) << shift) + ((1u << shift) >> 1);
          return weigh.one(value_of(bhi - min(off, bspan)));
        };
        auto count_of = [&](int e) {
          return (int)(e == 0 ? h[0] : e == 1 ? h[1] : e == 2 ? h[2] : h[3]);
        };
        Sum2 sum{0.f, 0.f}, in;
        if (h[0] | h[1] | h[2] | h[3]) {
#pragma unroll 1
          for (int e = 0; e < 4; ++e)
            if (count_of(e)) sum = sum_of(sum, times(weight_of(e), (float)count_of(e)));
        }
        if (lists) {
          const unsigned long long x = ranked(have, t < have ? s_list[t] : 0ull);
          const Sum2 w = t < have ? weigh.one(value_of((uint32_t)(x >> 32))) : Sum2{0.f, 0.f};
          const Sum2 before = sum_of(above, pairs_before(w, &in));
          // The first at which the target is reached is the last that is kept.
          if (t < have && !exceeds(target, sum_of(before, w))) atomicMin(&s_i[0], t);
          __syncthreads();
          const int last = s_i[0];
          if (last < have) {
            border = (uint32_t)(s_list[last] >> 32);
            ties = 1;
            while (ties <= last && (uint32_t)(s_list[last - ties] >> 32) == border) ++ties;
            limited = last + 1 < have && (uint32_t)(s_list[last + 1] >> 32) == border;
            break;
          }
        }
        Sum2 before = lists ? target : sum_of(above, pairs_before(sum, &in));
        if (sum.hi > 0.f && exceeds(target, before) && !exceeds(target, sum_of(before, sum))) {
          int e = 0, m;
          for (;; ++e) {  // (the last one that has any, if the sums' rounding says none)
            m = count_of(e);
            const Sum2 w = weight_of(e), after = sum_of(before, times(w, (float)m));
            const bool last = e == 3 || (h[3] | (e < 2 ? h[2] : 0) | (e < 1 ? h[1] : 0)) == 0;
            if (m && (last || !exceeds(target, after))) {
              // So many of the key as it takes to come to the target.
              const Sum2 need = sum_of(target, Sum2{-before.hi, -before.lo});
              const int most = m;
              m = max(1, min(most, (int)ceilf(__fdividef(need.hi, w.hi))));
              while (m > 1 && !exceeds(target, sum_of(before, times(w, (float)(m - 1))))) --m;
              while (m < most && exceeds(target, sum_of(before, times(w, (float)m)))) ++m;
              // (The first, where the sums' rounding lets two threads find it.)
              atomicMin(&s_found, (uint32_t)(4 * t + e) << 21 | (uint32_t)m << 1 |
                                      ((shift > 0 ? most <= sa::LIST / 4 : m < most) ? 1u : 0u));
              break;
            }
            before = after;
          }
        }
        __syncthreads();
        const uint32_t found = s_found;
        const int b = found == NONE ? -1 : (int)(found >> 21);
        if (b >= 0 && shift == 0) {
          border = bhi - (uint32_t)b;
          ties = (int)(found >> 1 & 0xfffffu);
          limited = found & 1u;
          break;
        }
        if (b >= 0) {  // one bin to either side
          list = found & 1u;
          const uint32_t o0 = (uint32_t)max(b - 1, 0) << shift;
          const unsigned long long o1 = ((unsigned long long)(b + 2) << shift) - 1;
          blo = o1 >= bspan ? blo : ehi - (uint32_t)o1;
          bhi = ehi - min(o0, bspan);
        } else if (!exact) {  // its end, or below
          bhi = bspan >> 1 > 1u << shift ? blo + (1u << shift) : blo + (bspan >> 1);
          blo = min(max(key_of(vlo - reach), elo), bhi);
          reach *= 16.f;
        } else if (blo == elo) {
          // (The sums' rounding: the keys from elo on come to the target, as an earlier look
          // from below said, or they are all.)
          border = elo;
          dense = true;
          break;
        } else if (blo <= lowest) {  // below the bins, and min_p's border in them
          border = lowest;
          dense = true;
          break;
        } else {  // below the bins
          above = sum_of(above, in);
          dense = true;
          ehi = bhi = blo - 1;
          blo = min(max(key_of(vlo - reach), elo), bhi);
          reach *= 16.f;
          list = true;
        }
        // The next list is written into every CTA's s_list by all of them, and the last cluster
        // barrier came before this one was ranked: they meet once more where there was a list.
        // (Lists that nobody ranked, too long or of bins below the border, are not read after that
        // barrier; bins, sums and lengths alternate.)
        if (lists)
          sync();
        else
          __syncthreads();
      }
      summed = dense ? 0u : bhi;
    }
    if (!done && lowest > border) {
      border = lowest;
      limited = false;
    }
  }
  if (!done) {
    // ---- every warp's kept weight, and the token ----
    // Keys from `from` on count whole; where ties are cut, those at the border by number.
    const uint32_t from = border + (limited ? 1 : 0);
    const float at = value_of(border);
    int c = 0;
    if (summed == 0) {
      const float vfrom = limited && border == kmax ? INFINITY : value_of(from);
      Sums s;
      each([&](int, uint4 g) {
#pragma unroll
        for (int x = 0; x < GROUP / 2; ++x) {
          const float2 v = Lg::pair(g, x);
          float2 hi, q;
          weigh(v, &hi, &q);
          s.add(make_float2(v.x >= vfrom ? hi.x : 0.f, v.y >= vfrom ? hi.y : 0.f), q);
        }
      });
      mine = s.all();
      if (limited) c = count_ties();
    } else if (border <= summed) {
      const float vhi = value_of(summed);
      each([&](int i, uint4 g) {
        each_of(within(g, at, vhi), i, [&](raw l, int) {
          const float v = Lg::value(l);
          if (v == at && limited) {
            ++c;
          } else {
            mine = sum_of(mine, weigh.one(v));
          }
        });
      });
    }
    const int r = round & 1;
    {
      const Sum2 s = warp_sum(mine);
      const int in_warp = __reduce_add_sync(0xffffffffu, c);
      if (lane < C) {
        put(remote(&s_warp[r][0][seg_id], lane), s.hi, s.lo);
        put(remote(&s_cnt[seg_id], lane), in_warp);
      }
    }
    sync();
    const Sum2 tie = weigh.one(at);
    if (warp == 0) {  // the segment
      const int per = (segs + 31) / 32, seg0 = lane * per;
      int ties_here = 0;
      if (limited) {
#pragma unroll 1
        for (int i = seg0; i < min(seg0 + per, segs); ++i) ties_here += s_cnt[i];
        ties_here = ties - count_before(ties_here);  // to keep from here on
      }
      auto segment = [&](int i, int* left) {
        Sum2 v = {s_warp[r][0][i].x, s_warp[r][0][i].y};
        if (limited) {
          v = sum_of(v, times(tie, (float)max(0, min(*left, s_cnt[i]))));
          *left -= s_cnt[i];
        }
        return v;
      };
      Sum2 sum{0.f, 0.f};
      int left = ties_here;
#pragma unroll 1
      for (int i = seg0; i < min(seg0 + per, segs); ++i) sum = sum_of(sum, segment(i, &left));
      const Sum2 all = warp_sum(sum), aim = times(all, uu);
      Sum2 base{0.f, 0.f};
      const int l = find(sum, aim, &base);
      // Of that lane's: the first at which they exceed the aim, or the last with any.
      int owner = -1, owner_left = 0;
      Sum2 owner_base = base;
      left = __shfl_sync(0xffffffffu, ties_here, l);
#pragma unroll 1
      for (int i = l * per; i < min(l * per + per, segs); ++i) {
        const int now = left;
        const Sum2 v = segment(i, &left);
        if (v.hi > 0.f && (owner < 0 || !exceeds(base, aim))) {
          owner = i;
          owner_left = now;
          owner_base = base;
        }
        base = sum_of(base, v);
      }
      if (lane == 0) {
        s_i[0] = owner;
        s_i[1] = owner_left;
        s_pair[2] = make_float2(all.hi, all.lo);
        s_pair[3] = make_float2(aim.hi, aim.lo);
        s_pair[4] = make_float2(owner_base.hi, owner_base.lo);
      }
    }
    __syncthreads();
    total = Sum2{s_pair[2].x, s_pair[2].y};
    if (s_i[0] == seg_id) {
      // Its lanes, then the tokens of one.
      const int skip = max(0, s_i[1] - count_before(c));
      const Sum2 aim = {s_pair[3].x, s_pair[3].y};
      Sum2 v = mine;
      if (limited) v = sum_of(v, times(tie, (float)min(skip, c)));
      Sum2 base = {s_pair[4].x, s_pair[4].y};
      const int l = find(v, aim, &base);
      int keep = __shfl_sync(0xffffffffu, skip, l);
      const raw* const e = reinterpret_cast<const raw*>(part) + (warp * 32 + l) * own * GROUP;
      int token = -1;
#pragma unroll 1
      for (int i0 = 0; i0 < own * GROUP; i0 += 32) {
        const float x = i0 + lane < own * GROUP ? Lg::value(e[i0 + lane]) : -INFINITY;
        const bool is_tie = limited && x == at;
        const uint32_t all_ties = __ballot_sync(0xffffffffu, is_tie);
        const bool kept = is_tie ? __popc(all_ties & ((1u << lane) - 1)) < keep : x >= at;
        keep -= __popc(all_ties);
        Sum2 w = weigh.one(x);
        if (!kept) w = Sum2{0.f, 0.f};
        const uint32_t some = __ballot_sync(0xffffffffu, w.hi > 0.f);
        if (!some) continue;
        const Sum2 inc = warp_sums(w);
        const uint32_t hits = __ballot_sync(0xffffffffu, w.hi > 0.f && exceeds(sum_of(base, inc), aim));
        token = i0 + (hits ? __ffs(hits) - 1 : 31 - __clz((int)some));
        if (hits) break;
        base = sum_of(base, lane_of(inc, 31));
      }
      if (lane == 0) p.tokens[row] = first + (warp * 32 + l) * own * GROUP + token;
    }
    if (p.probs && limited) cut = find_cut(c);
  } else if (!alive && rank == 0 && t == 0) {
    p.tokens[row] = -1;
  }
  if (p.probs) {
    // 1 / total as two floats.
    const float i_hi = alive ? __frcp_rn(total.hi) : 0.f;
    const float i_lo = -i_hi * __fmaf_rn(total.lo, i_hi, __fmaf_rn(total.hi, i_hi, -1.f));
    float* const dst = p.probs + row * p.V;
    const raw* const e = reinterpret_cast<const raw*>(part);
    const float at = value_of(border);
#pragma unroll 2
    for (int i = 2 * t; i < n; i += 2 * sa::THREADS) {
      const float2 v = make_float2(Lg::value(e[i]), Lg::value(e[i + 1]));
      const int x = first + i;
      const bool a = alive && (v.x > at || (v.x == at && x <= cut));
      const bool b = alive && (v.y > at || (v.y == at && x + 1 <= cut));
      float2 o = make_float2(0.f, 0.f);
      if (__any_sync(0xffffffffu, a || b)) {
        float2 hi, q;
        weigh(v, &hi, &q);
        auto share = [&](float h, float q) {
          return __fmaf_rn(h, i_hi, __fmaf_rn(h, i_lo, __fmul_rn(__fmul_rn(h, q), i_hi)));
        };
        if (a) o.x = share(hi.x, q.x);
        if (b) o.y = share(hi.y, q.y);
      }
      if (x >= 0 && x < p.V) dst[x] = o.x;
      if (x + 1 >= 0 && x + 1 < p.V) dst[x + 1] = o.y;
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
  const size_t smem = (size_t)p.groups * sa::THREADS * 16;
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
  // 16-byte groups per thread (the first begins where the row's alignment has it begin).
  auto groups_of = [&](int cluster) {
    const long long threads = (long long)cluster * fa::sa::THREADS;
    return (((long long)V + 2 * group - 2) / group + threads - 1) / threads;
  };
  auto part_of = [&](int cluster) { return groups_of(cluster) * fa::sa::THREADS * 16; };
  if (part_of(fa::sa::CLUSTER) > fa::sa::SMEM_MAX) return FA_ERR_UNSUPPORTED;
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
  // CTAs per row, by a model of the clocks: 1.2 per element on the SM that has most of
  // them (1.6 where it has one CTA at a time to run), 8000 per wave, 1000 more for a
  // cluster's meetings.  Measured for 1, 2, 4 and 8: one row of 32000 27, 16, 15.9, 13.3 us;
  // 200 of 50257 30, 26, 38, 61; 512 of 32000 129, 105, 160, 298; 64 of 128000 (2, 4, 8)
  // 66, 50, 59.
  double best = 0;
  for (int c = 1; c <= fa::sa::CLUSTER; c *= 2) {
    if (part_of(c) > fa::sa::SMEM_MAX) continue;
    const int fits = part_of(c) + 46 * 1024 > 113 * 1024 ? 1 : 2;
    const double ctas = (double)rows * c, waves = ctas / (fits * sms);
    const double per_sm = ceil(ctas / sms) * (double)(groups_of(c) * group * fa::sa::THREADS);
    const double clocks = per_sm * (fits == 1 || ctas <= sms ? 1.6 : 1.2) +
                          (waves < 1 ? 1 : waves) * (c > 1 ? 9000 : 8000);
    if (best == 0 || clocks < best) {
      best = clocks;
      p.cluster = c;
    }
  }
  p.groups = (int)groups_of(p.cluster);
  cudaError_t e;
  if (dtype == FA_FP32)
    e = fa::launch_sample<float>(p, rows, stream);
  else if (dtype == FA_BF16)
    e = fa::launch_sample<__nv_bfloat16>(p, rows, stream);
  else
    e = fa::launch_sample<__half>(p, rows, stream);
  return fa::record_cuda_status(e, "sampling launch");
}
