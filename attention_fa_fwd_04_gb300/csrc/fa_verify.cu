// fa_verify.cu -- the accepted path of a drafted tree (fa_verify_tree), and the
// cache rows of that path moved together (fa_compact_tree).
//
// Verification.  Node 0 is the last decided token, p_s the target's
// distribution after node s, q_s the distribution node s's children were drawn
// from.  At a node, with residual r = p_s and mass Z = 1, its children are
// tried in index order: child c with token x is accepted if
//   u_c q_s(x) Z < r(x),
// and the walk goes on from it; else r <- max(r - Z q_s, 0), Z <- sum r.  Where
// no child is left the next token is drawn from r with u_0: the lowest token
// whose cumulative r exceeds u_0 sum r.  (One residual after another is the
// rule that keeps the output distributed as the target's own samples when
// several children are drawn independently.)  Without q the drafts are taken
// as chosen outright, q_s the indicator of x: Z <- Z - r(x), r(x) <- 0.
//
// The answers are whole numbers, so a sum that is off by a rounding can change
// one.  With 128000 tokens, fp32 sums would move about one border in a hundred
// draws; residuals and sums are therefore kept as pairs of floats (48 bits, by
// error-free sums and products, of which a pass over a row keeps 46), which costs a
// dozen fp32 operations per element where fp64 would be bound by the few fp64
// units.  After rejections the residual is the difference of p and c q: its error
// is 2^-46 of those, whatever mass Z is left, so borders are good to 2^-46 c / Z.
//
// Bound: two rows of V floats per sequence (the node where its walk stops, and
// nodes where more than one child is tried), once from HBM and for further
// rejected siblings from L2; in fact the latency of the passes over a row that
// the sequence with the most rejections needs one after another: 64 trees of 32
// nodes over 128000 tokens take 34.5 us (1.9 TB/s of the rows where they stop; at
// most five passes of 6000 to 8000 clocks: the first loads' latency 1000, the
// walk 800 to 1900, the sums' meeting 900), one chain of 5 over 32000 tokens 5.2 us.
// The tests themselves
// read single elements: those of all nodes are fetched at once, and the walk
// runs on shared memory, in one warp of each CTA.  A cluster of up to 8 CTAs
// takes one sequence: every CTA walks (the same way), and for a mass each sums
// its part of the row and pushes its sum to the others, onto a barrier that
// counts the sums (2 us less than with a cluster barrier after each pass, 1150 clocks).
#include <math.h>

#include "fa.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

__device__ unsigned int g_verify_err = 0;

namespace vf {
constexpr int CLUSTER = 8;  // CTAs per sequence, at most
constexpr int SM_WARPS = 32;  // resident per SM, as two blocks of 16 warps or four of 8
constexpr int MAX_N = 64;
}  // namespace vf

struct VerifyParams {
  const float* p;  // [B, N, V]
  const float* q;  // [B, N, V] or null
  const int32_t* tokens;
  const int32_t* parents;
  const float* u;
  int32_t* path;
  int32_t* count;
  int32_t* next;
  int N, V;
  int cluster;  // CTAs per sequence
  int part;     // tokens per warp, a multiple of 128
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A probability as it counts: anything but a positive finite number is 0.
__device__ __forceinline__ float clean(float x) {
  return __float_as_uint(x) < 0x7f800000u ? x : 0.f;
}

// Unevaluated sum of two floats, |lo| at most half a step of hi.
struct __align__(8) Pair {
  float hi, lo;
};
// A store into CTA `rank` of the cluster that counts on that CTA's barrier, both
// given by this CTA's addresses.
__device__ __forceinline__ void store_remote(Pair* local, uint64_t* bar, uint32_t rank, Pair v) {
  asm volatile(
      "{\n\t.reg .b32 a, m;\n\t"
      "mapa.shared::cluster.u32 a, %0, %2;\n\t"
      "mapa.shared::cluster.u32 m, %1, %2;\n\t"
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [a], {%3, %4}, [m];\n\t}" ::"r"(
          smem_u32(local)),
      "r"(smem_u32(bar)), "r"(rank), "f"(v.hi), "f"(v.lo)
      : "memory");
}
// Until a barrier's phase is complete: polls, which a sum from another SM ends
// within about a microsecond, then suspends, within the teardown limit.
__device__ __forceinline__ void peers_wait(uint64_t* bar, uint32_t parity) {
  for (int i = 0; i < 256; ++i)
    if (mbar_test_wait(smem_u32(bar), parity)) return;
  if (!mbar_wait_drain(bar, parity)) atomicOr(&g_verify_err, kErrTimeout | (23u << 8));
}
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// |a| >= |b|.
__device__ __forceinline__ Pair fast_two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return fast_two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  const float h = __fmul_rn(a.hi, b.hi);
  float l = __fmaf_rn(a.hi, b.hi, -h);
  l = __fmaf_rn(a.hi, b.lo, l);
  return fast_two_sum(h, __fmaf_rn(a.lo, b.hi, l));
}
__device__ __forceinline__ bool above(Pair a, Pair b) {
  const Pair d = two_sum(a.hi, -b.hi);
  return __fadd_rn(d.hi, __fadd_rn(d.lo, __fsub_rn(a.lo, b.lo))) > 0.f;
}
__device__ __forceinline__ Pair shfl_up(Pair a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
}
__device__ __forceinline__ Pair shfl_xor(Pair a, int o) {
  return {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
}
__device__ __forceinline__ Pair shfl(Pair a, int l) {
  return {__shfl_sync(0xffffffffu, a.hi, l), __shfl_sync(0xffffffffu, a.lo, l)};
}
// max(p - c q, 0).
__device__ __forceinline__ Pair residual(float p, Pair c, float q) {
  const float h = __fmul_rn(c.hi, q);
  const float l = __fmaf_rn(c.lo, q, __fmaf_rn(c.hi, q, -h));
  Pair d = two_sum(p, -h);
  d = fast_two_sum(d.hi, __fsub_rn(d.lo, l));
  return d.hi > 0.f ? d : Pair{0.f, 0.f};
}

// The same on two elements at once (packed fp32 operations).
struct Pair2 {
  float2 hi, lo;
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  return __ffma2_rn(b, both(-1.f), a);
}
__device__ __forceinline__ Pair2 two_sum2(float2 a, float2 b) {
  const float2 s = __fadd2_rn(a, b), t = sub2(s, a);
  return {s, __fadd2_rn(sub2(a, sub2(s, t)), sub2(b, t))};
}
// max(p - c q, 0), as a pair whose lower part need not be below half a step.
// Where the difference counts, p is at least the rounded product, and its
// rounding error takes two more subtractions.  ONE: c = 1.
template <bool ONE>
__device__ __forceinline__ Pair2 residual2(float2 p, Pair c, float2 q) {
  Pair2 r;
  float2 sum;
  if constexpr (ONE) {
    r.hi = sub2(p, q);
    r.lo = sub2(sub2(p, r.hi), q);
    sum = r.hi;
  } else {
    const float2 nh = __fmul2_rn(both(-c.hi), q);
    const float2 l = __ffma2_rn(both(c.lo), q, __ffma2_rn(both(c.hi), q, nh));
    r.hi = __fadd2_rn(p, nh);
    r.lo = sub2(sub2(nh, sub2(r.hi, p)), l);
    sum = __fadd2_rn(r.hi, r.lo);
  }
  if (!(sum.x > 0.f)) r.hi.x = r.lo.x = 0.f;
  if (!(sum.y > 0.f)) r.hi.y = r.lo.y = 0.f;
  return r;
}

// What a node's n rejected children left of its row: with q, max(p - c q, 0),
// c = 1 + Z_1 + ... + Z_{n-1} the sum of the masses so far (taking Z q off an
// earlier residual again only lowers the same difference); without, p with the
// rejected tokens' entries 0.
struct Rejected {
  int n;
  Pair c;
  const int* token;
};

// Four elements of a row from v on: v, v + ST, v + 2 ST, v + 3 ST.  (ST = 1 by
// one 16-byte load where rows are aligned, else scalar loads, for a whole
// warp's group of 128 with ST = 32.)
template <bool VEC, int ST>
__device__ __forceinline__ float4 load4(const float* row, int v, int end) {
  if constexpr (VEC) {
    return v < end ? *reinterpret_cast<const float4*>(row + v) : make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    return make_float4(v < end ? row[v] : 0.f, v + ST < end ? row[v + ST] : 0.f,
                       v + 2 * ST < end ? row[v + 2 * ST] : 0.f,
                       v + 3 * ST < end ? row[v + 3 * ST] : 0.f);
  }
}
__device__ __forceinline__ float4 clean4(float4 a) {
  return make_float4(clean(a.x), clean(a.y), clean(a.z), clean(a.w));
}
// The largest of the four's bits: below those of infinity if all of them are
// probabilities as they stand.
__device__ __forceinline__ uint32_t bits4(float4 a) {
  return max(max(__float_as_uint(a.x), __float_as_uint(a.y)),
             max(__float_as_uint(a.z), __float_as_uint(a.w)));
}
// What is left of four clean elements.  LEVEL: rj.n where it is 0 or 1, else 2.
template <bool DRAFT, int ST, int LEVEL>
__device__ __forceinline__ void left4(float4 a, float4 d, int v, const Rejected& rj,
                                      Pair2 (&r)[2]) {
  r[0] = {make_float2(a.x, a.y), both(0.f)};
  r[1] = {make_float2(a.z, a.w), both(0.f)};
  if constexpr (LEVEL == 0) {
  } else if constexpr (DRAFT) {
    r[0] = residual2<LEVEL == 1>(r[0].hi, rj.c, make_float2(d.x, d.y));
    r[1] = residual2<LEVEL == 1>(r[1].hi, rj.c, make_float2(d.z, d.w));
  } else {
    for (int k = 0; k < rj.n; ++k) {
      const int o = rj.token[k] - v;
      if (o == 0) r[0].hi.x = 0.f;
      if (o == ST) r[0].hi.y = 0.f;
      if (o == 2 * ST) r[1].hi.x = 0.f;
      if (o == 3 * ST) r[1].hi.y = 0.f;
    }
  }
}

// A sum whose lower part may pass half a step of the upper one: a few of them
// may be added up so, and tidy() ends such a run.  (A third fewer operations in a
// row; 64 trees over 128000 tokens without q 20.6 -> 19.9 us.)
__device__ __forceinline__ Pair add_loose(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return {s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo))};
}
__device__ __forceinline__ Pair tidy(Pair a) { return fast_two_sum(a.hi, a.lo); }
__device__ __forceinline__ Pair lane_sum(const Pair2& a) {
  return add_loose({a.hi.x, a.lo.x}, {a.hi.y, a.lo.y});
}
__device__ __forceinline__ Pair warp_sum(Pair t) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t = add_loose(t, shfl_xor(t, o));
  return tidy(t);
}
__device__ __forceinline__ void gather(Pair2& acc, const Pair2 (&r)[2]) {
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const Pair2 s = two_sum2(acc.hi, r[e].hi);
    acc = {s.hi, __fadd2_rn(acc.lo, __fadd2_rn(s.lo, r[e].lo))};
  }
}

// Sum of what is left in [va, vb) of a row, over the warp, by loads into
// registers, four tokens per lane and 128: 16 bytes at once where rows are aligned
// (VEC).  LEVEL as in left4.  All loads of an iteration come before its sums: 512
// tokens of p, or 256 of p and of q (64 trees of 32 nodes, 128000 tokens: 34.5 us,
// half as many 43.5; a ring of bulk copies per warp, three iterations ahead, 42.8:
// a copy's latency is longer than a load's, and a pass is too short to hide it).
template <bool DRAFT, bool VEC, int LEVEL>
__device__ __forceinline__ Pair sum_loads(const float* pr, const float* qr, int va, int vb,
                                          const Rejected& rj) {
  constexpr bool use_q = DRAFT && LEVEL > 0;
  constexpr int ST = VEC ? 1 : 32;  // the lane's tokens: side by side, or every 32nd
  constexpr int G = use_q ? 2 : 4;
  Pair2 acc[2] = {{both(0.f), both(0.f)}, {both(0.f), both(0.f)}};
  for (int v = va + (threadIdx.x & 31) * (VEC ? 4 : 1); v < vb; v += 128 * G) {
    float4 a[G], d[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      a[g] = load4<VEC, ST>(pr, v + 128 * g, vb);
      d[g] = use_q ? load4<VEC, ST>(qr, v + 128 * g, vb) : a[g];
    }
    uint32_t top = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) top = max(top, use_q ? max(bits4(a[g]), bits4(d[g])) : bits4(a[g]));
    if (top >= 0x7f800000u) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        a[g] = clean4(a[g]);
        d[g] = clean4(d[g]);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      Pair2 r[2];
      left4<DRAFT, ST, LEVEL>(a[g], d[g], v + 128 * g, rj, r);
      gather(acc[g & 1], r);
    }
  }
  return warp_sum(add_loose(lane_sum(acc[0]), lane_sum(acc[1])));
}

// Whole warp: inclusive sums of n <= 32 values, one per lane.
__device__ __forceinline__ Pair scan(Pair x, int n) {
  const int lane = threadIdx.x & 31;
  for (int o = 1; o < n; o <<= 1) {
    const Pair y = shfl_up(x, o);
    if (lane >= o) x = add(y, x);
  }
  return x;
}
// Whole warp: which of n sums (in shared memory) the aim falls in: the first
// whose cumulative sum, on top of *before, exceeds it; else (u of 1, or the
// last rounding) the last that holds anything.  *before moves up to its start.
__device__ __forceinline__ int pick_part(const Pair* sums, int n, Pair aim, Pair* before) {
  const int lane = threadIdx.x & 31;
  const Pair s = lane < n ? sums[lane] : Pair{0.f, 0.f};
  const Pair inc = scan(s, n);
  const uint32_t some = __ballot_sync(0xffffffffu, s.hi > 0.f);
  const uint32_t past = __ballot_sync(0xffffffffu, above(add(*before, inc), aim)) & some;
  const int at = past ? __ffs(past) - 1 : 31 - __clz(some);
  const Pair up = shfl(inc, at > 0 ? at - 1 : 0);
  if (at > 0) *before = add(*before, up);
  return at;
}

// VEC: rows are 16-byte aligned (V a multiple of 4).  W: warps per CTA.
template <bool DRAFT, bool VEC, int W>
__global__ void __launch_bounds__(W * 32, vf::SM_WARPS / W)
    verify_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ int s_parent[vf::MAX_N], s_token[vf::MAX_N], s_rej[vf::MAX_N];
  __shared__ float s_u[vf::MAX_N], s_px[vf::MAX_N], s_qx[vf::MAX_N];
  __shared__ Pair s_warp[W];
  __shared__ Pair s_cta[2][vf::CLUSTER];
  __shared__ int s_pick[2][W];
  __shared__ int s_cur, s_nrej;
  __shared__ bool s_last, s_known;
  __shared__ uint64_t s_path;
  __shared__ uint32_t s_first[2];
  __shared__ Pair s_c;
  __shared__ uint64_t s_sums[2];  // counts the sums that arrive in s_cta
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank(), CL = p.cluster;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&s_sums[i], 1);
    fence_mbar_init();
    for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&s_sums[i], CL * sizeof(Pair));
  }
  __syncwarp();
  cluster_arrive();  // (waited for below: no CTA is written to before it runs)
  pdl_wait_primary();
  const int b = blockIdx.x / CL;
  const int N = p.N, V = p.V;
  const size_t node0 = (size_t)b * N;
  if (tid < N) {
    // Node tid: an edge that the walk may take, or parent -2.
    int par = tid == 0 ? -1 : p.parents[node0 + tid];
    const int x = p.tokens[node0 + tid];
    s_u[tid] = p.u[node0 + tid];
    if (tid > 0 && (par < -2 || par >= tid || (par >= 0 && (x < 0 || x >= V)))) {
      par = -2;
      if (rank == 0) atomicOr(&g_verify_err, kErrBounds);
    }
    const bool edge = tid > 0 && par >= 0;
    s_parent[tid] = edge ? par : -2;
    s_token[tid] = x;
    const float px = edge ? clean(p.p[(node0 + par) * V + x]) : 0.f;
    const float qx = DRAFT ? (edge ? clean(p.q[(node0 + par) * V + x]) : 0.f) : 1.f;
    s_px[tid] = px;
    s_qx[tid] = qx;
  }
  __syncthreads();
  if (tid < vf::MAX_N) {
    // Every node's test as a first child (Z = 1).
    const bool yes =
        tid < N && above(Pair{s_px[tid], 0.f}, mul(Pair{s_u[tid], 0.f}, Pair{s_qx[tid], 0.f}));
    const uint32_t w = __ballot_sync(0xffffffffu, yes);
    if (lane == 0) s_first[warp] = w;
  }
  __syncthreads();
  cluster_wait();

  int pass = 0;
  // Sum of what is left of node cur's row: s_warp, and s_cta[pass & 1].  All
  // threads of the cluster.
  auto mass_of = [&](int cur, const Rejected& rj) {
    const long long v0 = ((long long)rank * W + warp) * p.part;
    const int va = v0 < V ? (int)v0 : V, vb = v0 + p.part < V ? (int)(v0 + p.part) : V;
    const float* pr = p.p + (node0 + cur) * V;
    const float* qr = DRAFT ? p.q + (node0 + cur) * V : nullptr;
    const Pair s = rj.n == 0   ? sum_loads<DRAFT, VEC, 0>(pr, qr, va, vb, rj)
                   : rj.n == 1 ? sum_loads<DRAFT, VEC, 1>(pr, qr, va, vb, rj)
                               : sum_loads<DRAFT, VEC, 2>(pr, qr, va, vb, rj);
    if (lane == 0) s_warp[warp] = s;
    __syncthreads();
    ++pass;
    if (warp == 0) {
      Pair t = lane < W ? s_warp[lane] : Pair{0.f, 0.f};
#pragma unroll 1
      for (int o = W / 2; o > 0; o >>= 1) t = add_loose(t, shfl_xor(t, o));
      t = tidy(t);
      if (lane < CL) store_remote(&s_cta[pass & 1][rank], &s_sums[pass & 1], lane, t);
    }
    // The other CTAs' sums.  (All of them come: what a CTA waits for before it
    // sends is bounded, and all walk by the same sums.)  A CTA sends its next one
    // after this one has been read here, so two buffers are enough.
    peers_wait(&s_sums[pass & 1], ((pass - 1) >> 1) & 1);
    if (tid == 0) mbar_arrive_expect_tx(&s_sums[pass & 1], CL * sizeof(Pair));
  };
  // (The same bits in every warp of every CTA.)
  auto total_of = [&]() {
    Pair t = lane < CL ? s_cta[pass & 1][lane] : Pair{0.f, 0.f};
#pragma unroll 1
    for (int o = vf::CLUSTER / 2; o > 0; o >>= 1) t = add_loose(t, shfl_xor(t, o));
    return shfl(tidy(t), 0);
  };

  // The walk, by warp 0; the others join for masses.
  const int par0 = lane < N ? s_parent[lane] : -2, par1 = lane + 32 < N ? s_parent[lane + 32] : -2;
  auto children = [&](int node) {
    return (uint64_t)__ballot_sync(0xffffffffu, par0 == node) |
           (uint64_t)__ballot_sync(0xffffffffu, par1 == node) << 32;
  };
  int cur = 0, n_sum = -1;  // n_sum: rejections that the sums stand for
  Rejected rj{0, {0.f, 0.f}, s_rej};
  uint64_t path = 1, kids = warp == 0 ? children(0) : 0;
  Pair Z{1.f, 0.f};
  const uint64_t first_yes = s_first[0] | (uint64_t)s_first[1] << 32;
  for (;;) {
    if (warp == 0) {
      while (kids) {
        if (DRAFT && rj.n > 0) {
          if (n_sum != rj.n) break;
          Z = total_of();
        }
        const int c = __ffsll((long long)kids) - 1;
        kids &= kids - 1;
        Pair r{s_px[c], 0.f};
        bool yes;
        if (rj.n == 0) {
          yes = first_yes >> c & 1;
        } else {
          if constexpr (DRAFT) {
            r = residual(r.hi, rj.c, s_qx[c]);
          } else {
            for (int i = 0; i < rj.n; ++i)
              if (s_rej[i] == s_token[c]) r.hi = 0.f;
          }
          yes = above(r, mul(mul(Pair{s_u[c], 0.f}, Pair{s_qx[c], 0.f}), Z));
        }
        if (yes) {
          cur = c;
          path |= 1ull << c;
          kids = children(c);
          rj.n = 0;
          rj.c = {0.f, 0.f};
          n_sum = -1;
          Z = {1.f, 0.f};
        } else {
          if constexpr (DRAFT) {
            rj.c = add(rj.c, Z);
          } else {
            if (lane == 0) s_rej[rj.n] = s_token[c];
            __syncwarp();
            Z = add(Z, Pair{-r.hi, 0.f});
          }
          ++rj.n;
        }
      }
      if (lane == 0) {
        s_cur = cur;
        s_nrej = rj.n;
        s_c = rj.c;
        s_last = kids == 0;
        s_known = n_sum == rj.n;
        s_path = path;
      }
    }
    __syncthreads();
    const bool last = s_last, known = s_known;
    cur = s_cur;
    rj.n = s_nrej;
    rj.c = s_c;
    if (!known) mass_of(cur, rj);
    n_sum = rj.n;
    if (last) break;
  }

  if (rank == 0 && tid < N) {
    // Node k of the path: the k-th set bit.
    uint64_t m = s_path;
    const int n = __popcll(m);
    for (int i = 0; i < tid && m; ++i) m &= m - 1;
    p.path[node0 + tid] = m ? __ffsll((long long)m) - 1 : -1;
    if (tid == 0) p.count[b] = n;
  }

  // The next token.
  Pair total = total_of();
  if (!(total.hi > 0.f) && rj.n > 0) {  // nothing left: the target's own row
    rj.n = 0;
    mass_of(cur, rj);
    total = total_of();
  }
  auto draw = [&]() {
    if (!(total.hi > 0.f)) {
      if (rank == 0 && tid == 0) p.next[b] = -1;
      return;
    }
    const Pair aim = mul(Pair{s_u[0], 0.f}, total);
    Pair before{0.f, 0.f};
    if (pick_part(s_cta[pass & 1], CL, aim, &before) != rank) return;
    const int at = pick_part(s_warp, W, aim, &before);
    // That part of the row, a group of 128 tokens per warp, four per lane.
    const long long v0 = ((long long)rank * W + at) * p.part;
    const int vb = v0 + p.part < V ? (int)(v0 + p.part) : V;
    const float* pr = p.p + (node0 + cur) * V;
    const float* qr = DRAFT ? p.q + (node0 + cur) * V : nullptr;
    int found = INT32_MAX, last_v = -1;
    for (int w0 = (int)v0; w0 < vb && found == INT32_MAX; w0 += 128 * W) {
      const int v = w0 + warp * 128 + lane * 4;
      const float4 a = clean4(load4<VEC, 1>(pr, v, vb));
      float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
      if (DRAFT && rj.n > 0) d = clean4(load4<VEC, 1>(qr, v, vb));
      Pair2 r2[2];
      left4<DRAFT, 1, 2>(a, d, v, rj, r2);
      const Pair r[4] = {fast_two_sum(r2[0].hi.x, r2[0].lo.x), fast_two_sum(r2[0].hi.y, r2[0].lo.y),
                         fast_two_sum(r2[1].hi.x, r2[1].lo.x), fast_two_sum(r2[1].hi.y, r2[1].lo.y)};
      const Pair own = add(add(r[0], r[1]), add(r[2], r[3]));
      const Pair inc = scan(own, 32);
      __syncthreads();  // (s_warp and s_pick have been read)
      if (lane == 31) s_warp[warp] = inc;
      __syncthreads();
      const Pair upto = scan(lane < W ? s_warp[lane] : Pair{0.f, 0.f}, W);
      Pair start = shfl(upto, warp > 0 ? warp - 1 : 0);
      start = warp > 0 ? add(before, start) : before;
      const uint32_t some = __ballot_sync(0xffffffffu, own.hi > 0.f);
      const uint32_t past = __ballot_sync(0xffffffffu, above(add(start, inc), aim)) & some;
      const int l = past ? __ffs(past) - 1 : (some ? 31 - __clz(some) : 0);
      const Pair up = shfl(inc, l > 0 ? l - 1 : 0);
      if (lane == l) {
        // The lane's first that passes the aim; its last with mass where
        // rounding (or a missing aim) leaves none.
        Pair run = l > 0 ? add(start, up) : start;
        int pick = -1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (r[e].hi > 0.f && (!past || pick < 0 || !above(run, aim))) pick = v + e;
          run = add(run, r[e]);
        }
        s_pick[0][warp] = past ? pick : INT32_MAX;
        s_pick[1][warp] = some ? pick : -1;
      }
      __syncthreads();
      for (int i = 0; i < W; ++i) {
        found = s_pick[0][i] < found ? s_pick[0][i] : found;
        last_v = s_pick[1][i] > last_v ? s_pick[1][i] : last_v;
      }
      before = add(before, shfl(upto, W - 1));
    }
    if (tid == 0) p.next[b] = found != INT32_MAX ? found : last_v;
  };
  // The other CTAs may leave from here on, and this one once they are here: none
  // is written to after it has gone, even if a call's inputs change under it and
  // its CTAs disagree on the walk.
  cluster_arrive();
  draw();
  __syncwarp();
  cluster_wait();
}

// ---------------------------------------------------------------------------
// Compaction.  Sequence b keeps the nodes path[b][0 .. count[b]) of the tree in
// its last N slots: the i-th of them moves to slot L - N + i, in K and V of
// every layer, and the length becomes L - N + count.
//
// HBM bound, and mostly latency: a few rows of Hkv * D elements per sequence
// and layer.  A thread owns one 16-byte column and loads eight rows before it
// stores them.  That is safe in place: the path rises, so no row is a source
// after it was a destination, and columns do not meet.
// ---------------------------------------------------------------------------
namespace cp {
constexpr int THREADS = 256;
constexpr int MAX_N = 64;
constexpr int AHEAD = 8;
}  // namespace cp

struct CompactParams {
  uint4* k;
  uint4* v;
  const int32_t* page_table;
  const int32_t* seqlens;
  const int32_t* path;
  const int32_t* count;
  int32_t* seqlens_out;  // null: moves only
  int N, cols;           // cols: 16-byte columns of a row
  int num_pages, page_size, max_pages;
  long long layer;       // 16-byte columns of a layer's pool
  int move;              // 0: lengths only
};

__global__ void __launch_bounds__(cp::THREADS)
    compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ long long s_src[cp::MAX_N], s_dst[cp::MAX_N];
  pdl_launch_dependents();
  pdl_wait_primary();
  const int b = blockIdx.z, t = threadIdx.x;
  const int L = p.seqlens[b], n = p.count[b];
  const long long cap = (long long)p.max_pages * p.page_size;
  const bool first = blockIdx.x == 0 && blockIdx.y == 0;
  bool bad = L > cap || n < 0 || n > p.N;
  const bool pad = L < p.N;
  if (!bad && !pad && t < n) {
    const int* path = p.path + (size_t)b * p.N;
    const int a = path[t];
    if (a < t || a >= p.N || (t > 0 && path[t - 1] >= a)) {
      bad = true;
    } else if (a != t) {
      const int base = L - p.N;
      const int32_t* table = p.page_table + (size_t)b * p.max_pages;
      long long row[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int slot = base + (e ? t : a), pg = slot / p.page_size;
        const int id = table[pg];
        bad |= id < 0 || id >= p.num_pages;
        row[e] = ((long long)id * p.page_size + (slot - pg * p.page_size)) * p.cols;
      }
      s_src[t] = row[0];
      s_dst[t] = row[1];
    } else {
      s_src[t] = s_dst[t] = 0;
    }
  }
  bad = __syncthreads_or(bad);
  if (first && t == 0) {
    if (bad) atomicOr(&g_verify_err, kErrBounds);
    if (p.seqlens_out) p.seqlens_out[b] = bad || pad ? L : L - p.N + n;
  }
  if (bad || pad || !p.move) return;
  int x = blockIdx.x * cp::THREADS + t;
  if (x >= 2 * p.cols) return;
  uint4* pool = (x < p.cols ? p.k : p.v) + blockIdx.y * p.layer;
  if (x >= p.cols) x -= p.cols;
  for (int i0 = 0; i0 < n; i0 += cp::AHEAD) {
    uint4 r[cp::AHEAD];
#pragma unroll
    for (int e = 0; e < cp::AHEAD; ++e)
      if (i0 + e < n && s_src[i0 + e] != s_dst[i0 + e]) r[e] = pool[s_src[i0 + e] + x];
#pragma unroll
    for (int e = 0; e < cp::AHEAD; ++e)
      if (i0 + e < n && s_src[i0 + e] != s_dst[i0 + e]) pool[s_dst[i0 + e] + x] = r[e];
  }
}

int read_verify_error(unsigned int* out, int reset) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_verify_err, sizeof(v));
  if (e != cudaSuccess) return e;
  if (reset && v) {
    const unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_verify_err, &z, sizeof(z));
    if (e != cudaSuccess) return e;
  }
  *out = v;
  return cudaSuccess;
}

}  // namespace fa

static bool al(const void* p, unsigned n) {
  return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

extern "C" int fa_verify_tree(const float* target_probs, const float* draft_probs,
                              const int32_t* tokens, const int32_t* parents,
                              const float* uniforms, int32_t* path, int32_t* count,
                              int32_t* next_token, int B, int N, int V, cudaStream_t stream) {
  if (B < 0 || N < 1 || V < 1) return FA_ERR_INVALID_ARG;
  if (N > fa::vf::MAX_N) return FA_ERR_UNSUPPORTED;
  if (B > INT32_MAX / fa::vf::CLUSTER || V > INT32_MAX / 2) return FA_ERR_INVALID_ARG;
  if (B == 0) return FA_OK;
  if (!al(target_probs, 4) || (draft_probs && !al(draft_probs, 4)) || !al(tokens, 4) ||
      !al(parents, 4) || !al(uniforms, 4) || !al(path, 4) || !al(count, 4) || !al(next_token, 4))
    return FA_ERR_INVALID_ARG;
  const fa::SetupDuringCapture setup;
  fa::VerifyParams p = {};
  p.p = target_probs;
  p.q = draft_probs;
  p.tokens = tokens;
  p.parents = parents;
  p.u = uniforms;
  p.path = path;
  p.count = count;
  p.next = next_token;
  p.N = N;
  p.V = V;
  // CTAs per sequence: 8, or as few of 8 warps as leave all of them resident at
  // once (64 sequences of 128000 tokens: 8 CTAs 34.5 us, 4 51.8 us), or twice
  // that where a warp's part would pass 1024 tokens (200 of 32000: 4 CTAs 19.7 us,
  // 2 22.1 us of 16 warps); and no more than give each warp 256 tokens.
  // 16 warps where the SMs are not filled and a warp's part stays above 512
  // tokens (8 sequences of 152064: 16 warps 20.4 us, 8 21.1 us; 16 of 50256: 16
  // warps 15.8 us, 8 14.5 us; one of 32000: 5.8 and 5.2 us).
  const int sms = fa::sm_count() > 0 ? fa::sm_count() : 148;
  auto part_of = [&](int cluster, int warps) {
    const int n = cluster * warps;
    return ((V + n - 1) / n + 127) / 128 * 128;
  };
  p.cluster = fa::vf::CLUSTER;
  while (p.cluster > 1 &&
         (part_of(p.cluster / 2, 8) <= 256 ||
          (long long)B * p.cluster > 8ll * sms ||
          ((long long)B * p.cluster > 4ll * sms && part_of(p.cluster / 2, 8) <= 1024)))
    p.cluster /= 2;
  const int warps =
      (long long)B * p.cluster <= sms && part_of(p.cluster, 16) > 512 ? 16 : 8;
  p.part = part_of(p.cluster, warps);
  const bool vec = V % 4 == 0 && al(target_probs, 16) && (!draft_probs || al(draft_probs, 16));
  const dim3 grid((unsigned)B * p.cluster);
  void (*const kernels[2][4])(fa::VerifyParams) = {
      {fa::verify_kernel<false, false, 8>, fa::verify_kernel<false, true, 8>,
       fa::verify_kernel<true, false, 8>, fa::verify_kernel<true, true, 8>},
      {fa::verify_kernel<false, false, 16>, fa::verify_kernel<false, true, 16>,
       fa::verify_kernel<true, false, 16>, fa::verify_kernel<true, true, 16>}};
  const cudaError_t e =
      fa::launch_dependent(kernels[warps == 16][(draft_probs ? 2 : 0) + (vec ? 1 : 0)], grid,
                           warps * 32, stream, p, p.cluster);
  return fa::record_cuda_status(e, "tree verification launch");
}

extern "C" int fa_compact_tree(void* kpages, void* vpages, const int32_t* page_table,
                               const int32_t* seqlens, const int32_t* path, const int32_t* count,
                               int32_t* seqlens_out, int layers, int B, int N, int Hkv,
                               int num_pages, int page_size, int max_pages, int D,
                               cudaStream_t stream) {
  if (layers < 0 || B < 0 || N < 1 || Hkv < 0 || num_pages < 0 || max_pages < 0)
    return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_INVALID_ARG;
  if (page_size < 32 || page_size % 32 != 0) return FA_ERR_INVALID_ARG;
  if (N > fa::cp::MAX_N) return FA_ERR_UNSUPPORTED;
  if (B > 65535 || layers > 65535 || Hkv > (1 << 20)) return FA_ERR_INVALID_ARG;
  if ((int64_t)max_pages * page_size > INT32_MAX) return FA_ERR_INVALID_ARG;
  if (B == 0) return FA_OK;
  if (!al(seqlens, 4) || !al(path, 4) || !al(count, 4) || !al(seqlens_out, 4))
    return FA_ERR_INVALID_ARG;
  if (max_pages > 0 && !al(page_table, 4)) return FA_ERR_INVALID_ARG;
  const bool rows = layers > 0 && Hkv > 0 && num_pages > 0;
  if (rows && (!al(kpages, 16) || !al(vpages, 16))) return FA_ERR_INVALID_ARG;
  if ((int64_t)num_pages * page_size > (1ll << 40) / (2 * D) / (Hkv ? Hkv : 1))
    return FA_ERR_INVALID_ARG;
  const fa::SetupDuringCapture setup;
  fa::CompactParams p = {};
  p.k = static_cast<uint4*>(kpages);
  p.v = static_cast<uint4*>(vpages);
  p.page_table = page_table;
  p.seqlens = seqlens;
  p.path = path;
  p.count = count;
  p.N = N;
  p.cols = Hkv * D / 8;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.layer = (long long)num_pages * page_size * p.cols;
  // Lengths updated in place are written by a launch of their own: the moving
  // blocks of a sequence all read its old length.
  const bool in_place = seqlens_out == seqlens;
  cudaError_t e = cudaSuccess;
  if (rows) {
    p.move = 1;
    p.seqlens_out = in_place ? nullptr : seqlens_out;
    const unsigned gx = (unsigned)((2 * p.cols + fa::cp::THREADS - 1) / fa::cp::THREADS);
    e = fa::launch_dependent(fa::compact_kernel, dim3(gx, layers, B), fa::cp::THREADS, stream, p);
  }
  if (e == cudaSuccess && (in_place || !rows)) {
    p.move = 0;
    p.seqlens_out = seqlens_out;
    e = fa::launch_dependent(fa::compact_kernel, dim3(1, 1, B), fa::cp::THREADS, stream, p);
  }
  return fa::record_cuda_status(e, "tree compaction launch");
}
