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
// draws; residuals and sums are therefore kept as pairs of floats (about 48
// bits, by error-free sums and products), which costs a dozen fp32 operations
// per element where fp64 would be bound by the few fp64 units.
//
// Bound: two rows of V floats per sequence (the node where its walk stops),
// once from HBM and for further rejected siblings from L2; for few sequences,
// latency.  The tests themselves read single elements: those of all nodes are
// fetched at once, and the walk itself runs on shared memory.  A cluster of 8
// CTAs takes one sequence: every CTA walks (the same way), and for a mass each
// sums an eighth of the row and pushes its sum to the other seven.
#include <math.h>

#include "fa.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

__device__ unsigned int g_verify_err = 0;

namespace vf {
constexpr int CLUSTER = 8;
constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
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
  int part;  // tokens per warp, a multiple of 128
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(double* local, uint32_t rank, double v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.f64 [a], %2;\n\t}" ::"r"(smem_u32(local)),
      "r"(rank), "d"(v)
      : "memory");
}

// A probability as it counts: anything but a positive finite number is 0.
__device__ __forceinline__ float clean(float x) { return x > 0.f && x < INFINITY ? x : 0.f; }

// Unevaluated sum of two floats, |lo| at most half a step of hi.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
// max(r - Z q, 0).
__device__ __forceinline__ Pair residual(Pair r, Pair Z, float q) {
  const float h = __fmul_rn(Z.hi, q);
  const float l = __fmaf_rn(Z.lo, q, __fmaf_rn(Z.hi, q, -h));
  Pair d = two_sum(r.hi, -h);
  d.lo = __fadd_rn(d.lo, __fsub_rn(r.lo, l));
  const float s = __fadd_rn(d.hi, d.lo);
  const float e = __fsub_rn(d.lo, __fsub_rn(s, d.hi));
  return s > 0.f ? Pair{s, e} : Pair{0.f, 0.f};
}

// What a node's rejected children left: the masses before each rejection
// (drafted from q), or the rejected tokens (no q).
struct Rejected {
  int n;
  const Pair* mass;
  const int* token;
};

template <bool DRAFT>
__device__ __forceinline__ Pair left_of(float p, float q, int v, const Rejected& rj) {
  Pair r{clean(p), 0.f};
  if constexpr (DRAFT) {
    const float qc = clean(q);
    for (int i = 0; i < rj.n; ++i) r = residual(r, rj.mass[i], qc);
  } else {
    for (int i = 0; i < rj.n; ++i)
      if (rj.token[i] == v) r.hi = 0.f;
  }
  return r;
}

// VEC: rows are 16-byte aligned (V a multiple of 4).
template <bool DRAFT, bool VEC>
__global__ void __cluster_dims__(vf::CLUSTER, 1, 1) __launch_bounds__(vf::THREADS, 2)
    verify_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ int s_parent[vf::MAX_N], s_token[vf::MAX_N], s_rej[vf::MAX_N];
  __shared__ float s_u[vf::MAX_N], s_px[vf::MAX_N], s_qx[vf::MAX_N];
  __shared__ Pair s_mass[vf::MAX_N];
  __shared__ double s_warp[vf::WARPS];
  __shared__ double s_cta[2][vf::CLUSTER];
  pdl_launch_dependents();
  cluster_arrive();  // (waited for below: no CTA is written to before it runs)
  pdl_wait_primary();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank();
  const int b = blockIdx.x / vf::CLUSTER;
  const int N = p.N, V = p.V;
  const size_t node0 = (size_t)b * N;

  if (tid < N) {
    // Node tid: an edge that the walk may take, or parent -2.
    int par = tid == 0 ? -1 : p.parents[node0 + tid];
    const int x = p.tokens[node0 + tid];
    if (tid > 0 && (par < -2 || par >= tid || (par >= 0 && (x < 0 || x >= V)))) {
      par = -2;
      if (rank == 0) atomicOr(&g_verify_err, kErrBounds);
    }
    s_parent[tid] = tid == 0 ? -1 : (par < 0 ? -2 : par);
    s_token[tid] = x;
    s_u[tid] = p.u[node0 + tid];
    s_px[tid] = par >= 0 && tid > 0 ? clean(p.p[(node0 + par) * V + x]) : 0.f;
    s_qx[tid] = DRAFT && par >= 0 && tid > 0 ? clean(p.q[(node0 + par) * V + x]) : 1.f;
  }
  __syncthreads();
  cluster_wait();

  // The walk.  Every warp of every CTA takes the same steps.
  const int par0 = lane < N ? s_parent[lane] : -2, par1 = lane + 32 < N ? s_parent[lane + 32] : -2;
  int cur = 0, n_path = 1;
  uint64_t on_path = 1;
  int n_rej = 0, n_sum = -1;  // rejections at cur; rejections that s_warp, s_cta stand for
  int pass = 0;
  const long long v0 = ((long long)rank * vf::WARPS + warp) * p.part;
  const int va = v0 < V ? (int)v0 : V, vb = v0 + p.part < V ? (int)(v0 + p.part) : V;

  // Sum of what is left at cur after n rejections, over all of the row.
  auto mass_of = [&](int n) {
    const Rejected rj{n, s_mass, s_rej};
    const float* pr = p.p + (node0 + cur) * V;
    const float* qr = DRAFT ? p.q + (node0 + cur) * V : nullptr;
    Pair acc{0.f, 0.f};
    auto add = [&](float a, float d, int v) {
      const Pair r = left_of<DRAFT>(a, d, v, rj);
      const Pair s = two_sum(acc.hi, r.hi);
      acc = {s.hi, __fadd_rn(acc.lo, __fadd_rn(s.lo, r.lo))};
    };
    if constexpr (VEC) {
#pragma unroll 4
      for (int v = va + lane * 4; v < vb; v += 128) {
        const float4 a = *reinterpret_cast<const float4*>(pr + v);
        const float4 d = DRAFT ? *reinterpret_cast<const float4*>(qr + v) : a;
        add(a.x, d.x, v);
        add(a.y, d.y, v + 1);
        add(a.z, d.z, v + 2);
        add(a.w, d.w, v + 3);
      }
    } else {
#pragma unroll 8
      for (int v = va + lane; v < vb; v += 32) add(pr[v], DRAFT ? qr[v] : 0.f, v);
    }
    double s = (double)acc.hi + (double)acc.lo;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();  // (s_warp of an earlier pass has been read)
    if (lane == 0) s_warp[warp] = s;
    __syncthreads();
    if (warp == 0 && lane < vf::CLUSTER) {
      double t = 0.0;
#pragma unroll
      for (int i = 0; i < vf::WARPS; ++i) t += s_warp[i];
      store_remote(&s_cta[pass & 1][rank], lane, t);
    }
    cluster_sync();
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < vf::CLUSTER; ++i) t += s_cta[pass & 1][i];
    ++pass;
    n_sum = n;
    return t;
  };

  for (;;) {
    uint64_t kids = (uint64_t)__ballot_sync(0xffffffffu, par0 == cur) |
                    (uint64_t)__ballot_sync(0xffffffffu, par1 == cur) << 32;
    n_rej = 0;
    n_sum = -1;
    double Z = 1.0;
    int down = -1;
    while (kids) {
      const int c = __ffsll((long long)kids) - 1;
      kids &= kids - 1;
      const int x = s_token[c];
      double r = (double)s_px[c], qx = (double)s_qx[c];
      if constexpr (DRAFT) {
        if (n_rej > 0) {
          if (n_sum != n_rej) Z = mass_of(n_rej);
          for (int i = 0; i < n_rej; ++i) {
            const double z = (double)s_mass[i].hi + (double)s_mass[i].lo;
            r = fmax(r - z * qx, 0.0);
          }
        }
      } else {
        for (int i = 0; i < n_rej; ++i)
          if (s_rej[i] == x) r = 0.0;
      }
      if ((double)s_u[c] * qx * Z < r) {
        down = c;
        break;
      }
      __syncthreads();  // (the lists are still being read)
      if (tid == 0) {
        s_mass[n_rej] = {(float)Z, (float)(Z - (double)(float)Z)};
        s_rej[n_rej] = x;
      }
      __syncthreads();
      ++n_rej;
      if constexpr (!DRAFT) Z -= r;
    }
    if (down < 0) break;
    cur = down;
    on_path |= 1ull << cur;
    ++n_path;
  }

  if (rank == 0 && tid < N) {
    // Node k of the path: the k-th set bit.
    uint64_t m = on_path;
    for (int i = 0; i < tid && m; ++i) m &= m - 1;
    p.path[node0 + tid] = m ? __ffsll((long long)m) - 1 : -1;
    if (tid == 0) p.count[b] = n_path;
  }

  // The next token.
  if (n_sum != n_rej) mass_of(n_rej);
  double total = 0.0;
#pragma unroll
  for (int i = 0; i < vf::CLUSTER; ++i) total += s_cta[(pass - 1) & 1][i];
  if (!(total > 0.0) && n_rej > 0) {  // nothing left: the target's own row
    n_rej = 0;
    total = mass_of(0);
  }
  if (!(total > 0.0)) {
    if (rank == 0 && tid == 0) p.next[b] = -1;
    return;
  }
  const double aim = (double)s_u[0] * total;
  // The CTA and warp whose part of the row the aim falls in: the first whose
  // cumulative sum exceeds it, else (u of 1, or the last rounding) the last
  // that holds anything.
  double before = 0.0, run = 0.0;
  int at = -1;
#pragma unroll
  for (int i = 0; i < vf::CLUSTER; ++i) {
    const double s = s_cta[(pass - 1) & 1][i];
    if (s > 0.0 && (at < 0 || !(run > aim))) {
      at = i;
      before = run;
    }
    run += s;
  }
  if (at != rank) return;
  run = before;
  at = -1;
#pragma unroll
  for (int i = 0; i < vf::WARPS; ++i) {
    const double s = s_warp[i];
    if (s > 0.0 && (at < 0 || !(run > aim))) {
      at = i;
      before = run;
    }
    run += s;
  }
  if (at != warp) return;
  const Rejected rj{n_rej, s_mass, s_rej};
  const float* pr = p.p + (node0 + cur) * V;
  const float* qr = DRAFT ? p.q + (node0 + cur) * V : nullptr;
  int found = -1, last = -1;
  for (int v = va; v < vb && found < 0; v += 32) {
    const int x = v + lane;
    Pair r{0.f, 0.f};
    if (x < vb) r = left_of<DRAFT>(pr[x], DRAFT ? qr[x] : 0.f, x, rj);
    double inc = (double)r.hi + (double)r.lo;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t some = __ballot_sync(0xffffffffu, r.hi > 0.f);
    const uint32_t past = __ballot_sync(0xffffffffu, before + inc > aim) & some;
    if (past) found = v + __ffs(past) - 1;
    if (some) last = v + 31 - __clz(some);
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) p.next[b] = found >= 0 ? found : last;
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

template <typename P>
static cudaError_t launch_dependent(void (*kernel)(P), dim3 grid, int threads, cudaStream_t stream,
                                    const P& p) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
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
  const int parts = fa::vf::CLUSTER * fa::vf::WARPS;
  p.part = ((V + parts - 1) / parts + 127) / 128 * 128;
  const bool vec = V % 4 == 0 && al(target_probs, 16) && (!draft_probs || al(draft_probs, 16));
  const dim3 grid((unsigned)B * fa::vf::CLUSTER);
  cudaError_t e;
  if (draft_probs)
    e = vec ? fa::launch_dependent(fa::verify_kernel<true, true>, grid, fa::vf::THREADS, stream, p)
            : fa::launch_dependent(fa::verify_kernel<true, false>, grid, fa::vf::THREADS, stream, p);
  else
    e = vec ? fa::launch_dependent(fa::verify_kernel<false, true>, grid, fa::vf::THREADS, stream, p)
            : fa::launch_dependent(fa::verify_kernel<false, false>, grid, fa::vf::THREADS, stream, p);
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
