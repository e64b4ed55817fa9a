// fa_pages.cu -- bookkeeping of a paged cache on the device: page table, free
// pages, slot map and positions from the sequences' old and new lengths
// (fa_update_pages), and K/V rows of packed tokens written to their slots
// (fa_write_pages).
//
// Update.  With pages(L) = max(ceil(L / page_size), shared pages) a sequence gives
// back table entries [pages(new), pages(old)) or takes entries [pages(old),
// pages(new)).  The free pages are a stack: what is given back goes on top, in
// order of sequence and entry, then sequences take from the top in order.  Where a
// sequence's growth ends is three prefix sums over the sequences (pages given
// back, pages taken, tokens), so nothing is done one after another.
//
// Bound: latency.  16 bytes per sequence and 8 per new token are nothing beside
// the chain: lengths, sums, a page id, a store.  One cluster of up to 8 CTAs does
// everything in one launch: every CTA makes the sums of all sequences for itself
// (in shared memory), a cluster barrier separates the reading of lengths and count
// from their writing in place, another the writing of the table from the tokens' reading of
// it, and the CTAs share the entries and tokens.  What is done in a row is done at once:
// with one token after another, each with its own way to its page, a step of 64 sequences
// took 6.2 us instead of 3.6, 256 sequences with 40000 new tokens 14.7 instead of 10.6.
//
// Write.  A copy: every row is read and written once, eight 16-byte loads per thread
// ahead of their stores.  65536 tokens of 8 heads (D = 128) take 78 us, 6.8 TB/s, a plain
// copy's rate; 64 tokens 2.8 us.
#include <type_traits>

#include "fa.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

__device__ unsigned int g_pages_err = 0;

namespace pg {
constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int CLUSTER = 8;
constexpr int MAX_B = 4096;  // seven words per sequence in shared memory
}  // namespace pg

struct UpdateParams {
  int32_t* table;
  const int32_t* old_lens;
  const int32_t* new_lens;
  const int32_t* shared;  // or null
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* lens_out;
  int32_t* count_out;
  int32_t* cu;
  int32_t* slots;
  int32_t* positions;
  int B, page_size, max_pages, max_free, max_new;
  int vec;  // slots and positions take 16-byte stores
};

__device__ __forceinline__ long long warp_scan(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// Inclusive sums of N quantities over the block, and the block's totals.  Every thread
// must call it; sums: N * WARPS entries, free again after the next barrier.
template <int N>
__device__ __forceinline__ void block_scan(long long (&v)[N], long long* sums, long long (&total)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_scan(v[i]);
  __syncthreads();
  if (lane == 31) {
#pragma unroll
    for (int i = 0; i < N; ++i) sums[N * warp + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    long long all = 0, before = 0;
#pragma unroll
    for (int w = 0; w < pg::WARPS; ++w) {
      if (w == warp) before = all;
      all += sums[N * w + i];
    }
    v[i] += before;
    total[i] = all;
  }
}

// The last of v[0 .. n) (rising) that is at most x; v[0] is.
__device__ __forceinline__ int last_at_most(const int* v, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(pg::THREADS, 1)
    update_pages_kernel(const __grid_constant__ UpdateParams p) {
  extern __shared__ int s_words[];
  __shared__ long long s_sums[3 * pg::WARPS];
  __shared__ int s_taken;
  const int n1 = p.B + 1;
  int* const s_old = s_words;           // old length
  int* const s_new = s_old + n1;        // length that holds afterwards
  int* const s_po = s_new + n1;         // pages of the old length
  int* const s_pn = s_po + n1;          // pages of the new one
  int* const s_rel = s_pn + n1;         // pages given back by the sequences before
  int* const s_need = s_rel + n1;       // pages taken by the sequences before
  int* const s_cu = s_need + n1;        // new tokens of the sequences before
  const int t = threadIdx.x;
  const int rank = (int)blockIdx.x, n_ctas = (int)gridDim.x;  // (the grid is one cluster)
  pdl_launch_dependents();
  pdl_wait_primary();
  if (t == 0) s_taken = 0;
  const long long cap = (long long)p.max_pages * p.page_size;
  const int F = *p.free_count;
  bool odd = false;
  // Pages given back, pages and tokens taken by all sequences before.
  long long all[3] = {0, 0, 0};
  for (int b0 = 0; b0 < p.B; b0 += pg::THREADS) {
    const int b = b0 + t;
    long long v[3] = {0, 0, 0}, total[3];
    if (b < p.B) {
      const int o = p.old_lens[b];
      int n = p.new_lens[b];
      const int sh = p.shared ? p.shared[b] : 0;
      const bool bad = o < 0 || n < 0 || o > cap || n > cap || sh < 0 || sh > p.max_pages;
      odd |= bad;
      int po = 0, pn = 0;
      if (bad) {
        n = o;
      } else {
        po = max((int)(((uint32_t)o + p.page_size - 1) / (uint32_t)p.page_size), sh);
        pn = max((int)(((uint32_t)n + p.page_size - 1) / (uint32_t)p.page_size), sh);
      }
      s_old[b] = o;
      s_new[b] = n;
      s_po[b] = po;
      s_pn[b] = pn;
      v[0] = max(po - pn, 0);
      v[1] = max(pn - po, 0);
      v[2] = max(n - o, 0);
    }
    const long long mine[3] = {v[0], v[1], v[2]};
    block_scan(v, s_sums, total);
    if (b < p.B) {
      int* const dst[3] = {s_rel, s_need, s_cu};
#pragma unroll
      for (int i = 0; i < 3; ++i) dst[i][b] = (int)min(all[i] + v[i] - mine[i], (long long)INT32_MAX);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) all[i] += total[i];
  }
  // A stack that is no stack, or that what comes back does not fit: nothing changes.
  const bool refuse = F < 0 || F > p.max_free || F + all[0] > p.max_free;
  odd |= refuse;
  if (odd && rank == 0) atomicOr(&g_pages_err, kErrBounds);
  const long long have = refuse ? 0 : F + all[0];
  long long cu0 = all[2];
  if (refuse || all[1] > have || all[2] > p.max_new) {
    // Not everything fits: which sequences do.
    long long need0 = 0, tok0 = 0;
    cu0 = 0;
    __syncthreads();
    for (int b0 = 0; b0 < p.B; b0 += pg::THREADS) {
      const int b = b0 + t;
      long long v[2] = {0, 0}, cu[1], v_all[2], cu_all[1];
      if (b < p.B) {
        if (refuse) {
          s_new[b] = s_old[b];
          s_pn[b] = s_po[b];
        }
        v[0] = max(s_pn[b] - s_po[b], 0);
        v[1] = max(s_new[b] - s_old[b], 0);
      }
      const long long my_need = v[0], my_tok = v[1];
      block_scan(v, s_sums, v_all);
      const long long need = need0 + v[0], tok = tok0 + v[1];
      const bool fits = (need <= have || my_need == 0) && tok <= p.max_new;
      cu[0] = fits ? my_tok : 0;
      const long long my_cu = cu[0];
      block_scan(cu, s_sums, cu_all);
      if (b < p.B) {
        s_need[b] = (int)min(need - my_need, (long long)INT32_MAX);
        s_cu[b] = (int)(cu0 + cu[0] - my_cu);
        if (!fits && my_tok > 0) {
          s_new[b] = s_old[b];
          s_pn[b] = s_po[b];
        } else if (my_need > 0) {
          atomicMax(&s_taken, (int)need);
        }
      }
      need0 += v_all[0];
      tok0 += v_all[1];
      cu0 += cu_all[0];
    }
  } else if (t == 0) {
    s_taken = (int)all[1];
  }
  const int tokens = (int)cu0;
  // Every CTA has read the lengths and the count, which may be written in place.
  if (n_ctas > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  __syncthreads();
  const int taken = s_taken;
  const int left = refuse ? F : (int)(have - taken);
  const int at = rank * pg::THREADS + t, step = n_ctas * pg::THREADS;
  // Page i of those given back, and the k-th page from the top of the stack.  (Rows
  // that give back are not written, nor are the free pages below F.)
  auto given = [&](int i) {
    const int b = last_at_most(s_rel, p.B, i);
    return p.table[(size_t)b * p.max_pages + s_pn[b] + (i - s_rel[b])];
  };
  auto taken_page = [&](int k) {
    const int i = (int)(have - 1 - k);
    return i < F ? p.free_pages[i] : given(i - F);
  };
  for (int b = at; b < p.B; b += step) {
    p.lens_out[b] = s_new[b];
    p.cu[b] = s_cu[b];
  }
  if (at == 0) {
    p.cu[p.B] = tokens;
    *p.count_out = left;
  }
  for (int k = at; k < taken; k += step) {
    const int b = last_at_most(s_need, p.B, k);
    p.table[(size_t)b * p.max_pages + s_po[b] + (k - s_need[b])] = taken_page(k);
  }
  // The tokens' pages are in the table, then: no searches among what was given back.
  auto arrive = [&] { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); };
  if (n_ctas > 1) arrive();
  // Four in a row, mostly of one sequence.
  for (long long i0 = F + 4ll * at; !refuse && i0 < left; i0 += 4ll * step) {
    int b = last_at_most(s_rel, p.B, (int)(i0 - F)), id[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = (int)(i0 - F) + e;
      if (i0 + e >= left) continue;
      while (i - s_rel[b] >= s_po[b] - s_pn[b]) ++b;
      id[e] = p.table[(size_t)b * p.max_pages + s_pn[b] + (i - s_rel[b])];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i0 + e < left) p.free_pages[i0 + e] = id[e];
  }
  if (n_ctas > 1)
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
  const int most = INT32_MAX / p.page_size;  // ids below it have 31-bit slots
  // A token per thread, or four in a row: one search, then all their table entries at once.
  auto tokens_of = [&](auto count) {
    constexpr int N = decltype(count)::value;
    for (long long t0 = (long long)N * at; t0 < p.max_new; t0 += (long long)N * step) {
      int slot[N], pos[N], id[N], first[N], b = 0;
      bool wants[N];  // (a token in a page that is not shared: those are not written)
      if (t0 < tokens) b = last_at_most(s_cu, p.B, (int)t0);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        pos[e] = first[e] = id[e] = 0;
        wants[e] = false;
        if (t0 + e < tokens) {
          const int x = (int)t0 + e;
          while (x - s_cu[b] >= s_new[b] - s_old[b]) ++b;  // the next sequence with new tokens
          pos[e] = s_old[b] + (x - s_cu[b]);
          const int page = (int)((uint32_t)pos[e] / (uint32_t)p.page_size);
          first[e] = page * p.page_size;
          wants[e] = !(p.shared && page < p.shared[b]);
          if (wants[e]) id[e] = p.table[(size_t)b * p.max_pages + page];
        }
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const bool fine = id[e] >= 0 && id[e] < most;
        slot[e] = wants[e] && fine ? id[e] * p.page_size + (pos[e] - first[e]) : -1;
        if (wants[e] && !fine) atomicOr(&g_pages_err, kErrBounds);
      }
      if constexpr (N == 4) {
        if (p.vec && t0 + 4 <= p.max_new) {
          *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
          *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
          continue;
        }
      }
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (t0 + e < p.max_new) {
          p.slots[t0 + e] = slot[e];
          p.positions[t0 + e] = pos[e];
        }
    }
  };
  if (p.max_new <= step)
    tokens_of(std::integral_constant<int, 1>{});
  else
    tokens_of(std::integral_constant<int, 4>{});
}

// Rows to slots: a thread takes AHEAD chunks of 16 bytes, of K and of V, all loads
// before the stores.
namespace wp {
constexpr int THREADS = 256;
constexpr int AHEAD = 4;
}  // namespace wp

struct WriteParams {
  const uint4* k;
  const uint4* v;
  uint4* kp;
  uint4* vp;
  const int32_t* slots;
  long long chunks;        // T * cols
  long long ks, vs;        // token strides in chunks
  long long slots_all;     // slots of the cache
  int cols;                // chunks of a row
};

template <bool WIDE>
__global__ void __launch_bounds__(wp::THREADS) write_pages_kernel(
    const __grid_constant__ WriteParams p) {
  pdl_launch_dependents();
  pdl_wait_primary();
  const long long base = (long long)blockIdx.x * (wp::THREADS * wp::AHEAD) + threadIdx.x;
  uint4 k[wp::AHEAD], v[wp::AHEAD];
  long long dst[wp::AHEAD];
  bool odd = false;
#pragma unroll
  for (int e = 0; e < wp::AHEAD; ++e) {
    const long long i = base + e * wp::THREADS;
    dst[e] = -1;
    if (i < p.chunks) {
      const long long tok = WIDE ? i / p.cols : (long long)((uint32_t)i / (uint32_t)p.cols);
      const int col = (int)(i - tok * p.cols);
      const int s = p.slots[tok];
      if (s >= 0 && s < p.slots_all) {
        dst[e] = (long long)s * p.cols + col;
        k[e] = p.k[tok * p.ks + col];
        v[e] = p.v[tok * p.vs + col];
      }
      odd |= s >= p.slots_all;
    }
  }
#pragma unroll
  for (int e = 0; e < wp::AHEAD; ++e)
    if (dst[e] >= 0) {
      p.kp[dst[e]] = k[e];
      p.vp[dst[e]] = v[e];
    }
  if (odd) atomicOr(&g_pages_err, kErrBounds);
}

int read_pages_error(unsigned int* out, int reset) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_pages_err, sizeof(v));
  if (e != cudaSuccess) return e;
  if (reset && v) {
    const unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_pages_err, &z, sizeof(z));
    if (e != cudaSuccess) return e;
  }
  *out = v;
  return cudaSuccess;
}

}  // namespace fa

static bool al(const void* p, unsigned n) {
  return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

extern "C" int fa_update_pages(int32_t* page_table, const int32_t* old_lens,
                               const int32_t* new_lens, const int32_t* shared_pages,
                               int32_t* free_pages, const int32_t* free_count, int32_t* lens_out,
                               int32_t* free_count_out, int32_t* cu_new, int32_t* slots,
                               int32_t* positions, int B, int page_size, int max_pages,
                               int max_free, int max_new, cudaStream_t stream) {
  if (B < 0 || max_pages < 0 || max_free < 0 || max_new < 0) return FA_ERR_INVALID_ARG;
  if (page_size < 32 || page_size % 32 != 0) return FA_ERR_INVALID_ARG;
  if ((int64_t)max_pages * page_size > INT32_MAX) return FA_ERR_INVALID_ARG;
  if (B > fa::pg::MAX_B) return FA_ERR_UNSUPPORTED;
  if (!al(free_count, 4) || !al(free_count_out, 4) || !al(cu_new, 4)) return FA_ERR_INVALID_ARG;
  if (B > 0 && (!al(old_lens, 4) || !al(new_lens, 4) || !al(lens_out, 4)))
    return FA_ERR_INVALID_ARG;
  if (shared_pages && !al(shared_pages, 4)) return FA_ERR_INVALID_ARG;
  if (B > 0 && max_pages > 0 && !al(page_table, 4)) return FA_ERR_INVALID_ARG;
  if (max_free > 0 && !al(free_pages, 4)) return FA_ERR_INVALID_ARG;
  if (max_new > 0 && (!al(slots, 4) || !al(positions, 4))) return FA_ERR_INVALID_ARG;
  const fa::SetupDuringCapture setup;
  fa::UpdateParams p = {};
  p.table = page_table;
  p.old_lens = old_lens;
  p.new_lens = new_lens;
  p.shared = shared_pages;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.lens_out = lens_out;
  p.count_out = free_count_out;
  p.cu = cu_new;
  p.slots = slots;
  p.positions = positions;
  p.B = B;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.max_free = max_free;
  p.max_new = max_new;
  p.vec = al(slots, 16) && al(positions, 16);
  const size_t smem = 7 * ((size_t)B + 1) * sizeof(int);
  static int attr_set[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= 64 || !__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE))) {
    e = cudaFuncSetAttribute(fa::update_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(7 * (fa::pg::MAX_B + 1) * sizeof(int)));
    if (e == cudaSuccess && dev >= 0 && dev < 64)
      __atomic_store_n(&attr_set[dev], 1, __ATOMIC_RELEASE);
  }
  if (e != cudaSuccess) return fa::record_cuda_status(e, "page update setup");
  int cluster = 1;
  while (cluster < fa::pg::CLUSTER && (long long)cluster * fa::pg::THREADS * 4 < max_new) cluster *= 2;
  e = fa::launch_dependent(fa::update_pages_kernel, dim3(cluster), fa::pg::THREADS, stream, p,
                           cluster, smem);
  return fa::record_cuda_status(e, "page update launch");
}

extern "C" int fa_write_pages(const void* k, const void* v, void* kpages, void* vpages,
                              const int32_t* slots, long long T, int Hkv, int num_pages,
                              int page_size, int D, long long k_stride, long long v_stride,
                              cudaStream_t stream) {
  if (T < 0 || Hkv < 0 || num_pages < 0) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_INVALID_ARG;
  if (page_size < 32 || page_size % 32 != 0) return FA_ERR_INVALID_ARG;
  if (T == 0 || Hkv == 0) return FA_OK;
  if (T > INT32_MAX || Hkv > (1 << 20)) return FA_ERR_INVALID_ARG;
  if (!al(k, 16) || !al(v, 16) || !al(slots, 4)) return FA_ERR_INVALID_ARG;
  if (num_pages > 0 && (!al(kpages, 16) || !al(vpages, 16))) return FA_ERR_INVALID_ARG;
  const long long row = (long long)Hkv * D;
  if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return FA_ERR_INVALID_ARG;
  if ((int64_t)num_pages * page_size > INT32_MAX) return FA_ERR_INVALID_ARG;
  const fa::SetupDuringCapture setup;
  fa::WriteParams p = {};
  p.k = static_cast<const uint4*>(k);
  p.v = static_cast<const uint4*>(v);
  p.kp = static_cast<uint4*>(kpages);
  p.vp = static_cast<uint4*>(vpages);
  p.slots = slots;
  p.cols = (int)(row / 8);
  p.chunks = T * p.cols;
  p.ks = k_stride / 8;
  p.vs = v_stride / 8;
  p.slots_all = (long long)num_pages * page_size;
  const long long per = fa::wp::THREADS * fa::wp::AHEAD, blocks = (p.chunks + per - 1) / per;
  if (blocks > INT32_MAX) return FA_ERR_INVALID_ARG;
  const cudaError_t e = fa::launch_dependent(
      p.chunks + per > 0xffffffffll ? fa::write_pages_kernel<true> : fa::write_pages_kernel<false>,
      dim3((unsigned)blocks), fa::wp::THREADS, stream, p);
  return fa::record_cuda_status(e, "page write launch");
}
