// fa_tree.cu -- attention of a tree of drafted tokens over a paged KV cache.
//
// What it computes: sequence b has L valid tokens, the last N of them the
// nodes of a tree (node s at position L - N + s, its parent a lower node).
// Query row (s, h) attends to the keys before the tree and to the nodes on its
// own way to the root, itself among them:
//   O = sum_j p_j V_j / sum_j p_j,  p_j = exp(scale <q, K_j> - max),
//   j < L - N, or j = L - N + a for an ancestor-or-self a of s.
//
// Floor: each K/V byte is read once per row tile, and serves N * G query rows
// (G = Hq / Hkv).  128 rows are 128 flops per byte, half of what the card
// needs to be matrix-bound, so up to about 256 rows per kv head the floor is the
// cache stream from HBM, and the matrix units above.  What bounds it at D = 128 and
// two to eight row tiles is near that (16 sequences of up to 16384 tokens, 256 rows,
// 134 us against 97.5; one of 65536, 1024 rows, 187 against 142); with one row tile
// per CTA (up to 128, 257 to 384 and 513 to 640 rows) and at D = 64 it is the softmax
// warps, 1.3 to 1.4e12 exponentials a second on one warpgroup per SM (4 sequences of
// up to 16000 tokens, 336 rows: 39 us at D = 128, 35 at D = 64, against 12 and 6),
// and over many short sequences each stretch's start and end.
//
// P is rounded to the inputs' type for P V: in fp32 it would need another kind of
// MMA, at half of the rate or less, twice the tensor memory, and V converted.  Each
// term of the sum is off by at most half a step of that type, relative to itself.
//
// Design: the rows (s, g) of one kv head are the M of tcgen05 MMAs against
// 128-key tiles of the paged cache (S = Q K^T and O += P V, both accumulated in
// tensor memory, P written back over S as PV's operand).
//   CTA = MT warpgroups of softmax (one 128-row tile each), one TMA producer
//   warp, one MMA warp.  MT = 1 (one, three or five row tiles): S is
//   double-buffered, so S of the next tile runs under this tile's softmax.
//   MT = 2: two row tiles share every K/V tile, one's MMAs under the other's
//   softmax.
// Split: lengths are device data.  All K/V tiles of all (sequence, kv head)
// units, with a few places after each for what a stretch costs beside its tiles,
// form one list, cut into equal ranges, one per group of n_rt CTAs (one
// CTA per row tile, side by side, so that they share K/V through L2).  A range
// may end inside a unit; its part of that unit goes to fp32 partials (O, max,
// sum) that a second kernel merges.  A unit inside one range is finished in
// place.  So every SM is busy for about the same time whatever the lengths, and a
// CTA writes at most two partials.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "fa.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_tiles.cuh"

namespace fa {

__device__ unsigned int g_tree_err = 0;

namespace tr {
using namespace tiles;
constexpr int MAX_N = 64;  // tree nodes: one 64-bit ancestor mask per row

template <int D, int MT>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE_BYTES = HALVES * HALF_BYTES;
  // MT = 2: three warpgroups, for the register split (setmaxnreg): launched with
  // 168 registers a thread, the softmax warpgroups take 208, the third keeps 88
  // (256 * 208 + 128 * 88 = 384 * 168, the launch's registers).  The compiler spills
  // 344 bytes of stores and 508 of loads there (MT = 1, 253 registers: none).
  static constexpr int THREADS = MT == 1 ? 192 : 384;
  static constexpr int RT = MT * BM;  // rows per CTA
  static constexpr int NSTAGE = D == 128 ? (MT == 1 ? 6 : 4) : 12;
  // MT = 2 (matrix-bound): ring positions 2g - 1 (a V) and 2g (the K after it)
  // share a pair of slots, released by one commit, and land on one barrier: the
  // MMA warp's instruction stream paces the kernel, and a commit or a wait
  // less per tile shows.  MT = 1 (bound by memory) releases slots one by one.
  static constexpr bool PAIRED = MT == 2;
  static constexpr int NPAIR = NSTAGE / 2;
  static_assert(NSTAGE % 2 == 0, "pairs");
  static constexpr int SMEM_Q = MT * TILE_BYTES;
  static constexpr int SMEM_KV = NSTAGE * TILE_BYTES;
  static constexpr int SMEM_BAR = 512;
  static constexpr int SMEM_TOTAL = 1024 + SMEM_Q + SMEM_KV + SMEM_BAR;
  static_assert(SMEM_TOTAL <= 227 * 1024, "shared memory per CTA");
  static_assert(NSTAGE / 2 + 2 < BAD_RING, "tiles in flight");
  // Tensor memory: two S buffers (MT = 1: of alternate tiles; MT = 2: of the
  // two row tiles), then O of each row tile.
  static constexpr uint32_t COL_S = 0, COL_O = 256, TMEM_COLS = 512;
};
}  // namespace tr

struct TreeParams {
  const void* q;  // [B, N, Hq, D]
  void* o;        // [B, N, Hq, D]
  float* lse;     // [B, N, Hq] or null
  const int32_t* page_table;
  const int32_t* seqlens;
  const int32_t* parents;  // [B, N]
  float* part_o;           // [CTAs][2][D / 4][rt_rows][4] unnormalised partial outputs
  float* part_ml;          // [CTAs][2][rt_rows][2] (max in log2 units, sum)
  long long* start;        // [B + 1] place of each sequence in the list, then the slack
  int B, N, Hq, Hkv, G, rows, rt_rows, n_rt, groups;
  int page_size, max_pages, num_pages, box;
  float c;  // scale * log2(e)
};

// Length of sequence b as the tree takes it: 0 for padding (fewer than N
// tokens) and for a length past the page table.
__device__ __forceinline__ int tree_len(const TreeParams& p, int b) {
  const int L = p.seqlens[b];
  return (L < p.N || (long long)L > (long long)p.max_pages * p.page_size) ? 0 : L;
}
__device__ __forceinline__ int tree_tiles(const TreeParams& p, int b) {
  return (int)(((uint32_t)tree_len(p, b) + tr::BN - 1) / tr::BN);  // (lengths reach 2^31 - 1)
}

// The list: the tiles of every unit (sequence, kv head), each unit's followed by
// `slack` places without a tile.  A stretch costs about that many tiles beside its
// own (Q, masks, the masked last tile, the epilogue), so equal shares of the list
// take about equal times: 16 sequences of up to 16384 tokens, 256 rows per kv head
// 132.8 us, without slack 140.4, with 2 places 138.1, with 8 135.8; 48 of up to
// 931, 2 rows 34.4, 39.1, 35.5 and 35.1.  Where there is no more than a tile per
// group there is no slack.
constexpr int kSlack = 4;

// A CTA's place in the list.
struct TreeWalk {
  long long x, hi;  // next and last place of the range
  long long first;  // first place of sequence b
  int b, T;         // sequence and its tiles per kv head
  int slack;
  __device__ __forceinline__ int places() const { return T > 0 ? T + slack : 0; }
};
struct TreeSeg {
  int b, hkv, t0, n, T, L;
};

// Groups in use: every one of them has a place (a group without one between two
// of a unit's would leave the merge a partial that nobody wrote).
__device__ __forceinline__ long long tree_groups(const TreeParams& p, long long total) {
  return total < p.groups ? total : p.groups;
}

// Whole warp: the range of group g and the sequence it starts in.
__device__ TreeWalk tree_plan(const TreeParams& p, int g) {
  const int lane = threadIdx.x & 31;
  TreeWalk w;
  w.first = 0;
  w.b = 0;
  w.T = 0;
  // tiles: per kv head, of the n sequences that have any.
  auto range = [&](long long tiles, int n) {
    w.slack = tiles * p.Hkv > p.groups ? kSlack : 0;
    const long long total = (tiles + (long long)n * w.slack) * p.Hkv;
    const long long G = tree_groups(p, total);
    w.x = g < G ? mul_div(total, g, G) : 0;
    w.hi = g < G ? mul_div(total, g + 1, G) : 0;
    return w.x < w.hi;
  };
  // The sequence of lane l (tiles T, inclusive places inc on top of `before`) is
  // the first that ends past the range's start.
  auto find = [&](int b0, int T, long long inc, long long before) {
    const uint32_t past = __ballot_sync(0xffffffffu, w.x < (before + inc) * p.Hkv);
    if (!past) return false;
    const int l = __ffs(past) - 1;
    w.b = b0 + l;
    w.T = __shfl_sync(0xffffffffu, T, l);
    w.first = (before + __shfl_sync(0xffffffffu, inc, l) - w.places()) * p.Hkv;
    return true;
  };
  const uint32_t upto = 0xffffffffu >> (31 - lane);  // lanes up to this one
  if (p.B <= 32) {  // one load, 32-bit sums (a sequence has at most 2^24 tiles)
    const int T = lane < p.B ? tree_tiles(p, lane) : 0;
    const uint32_t some = __ballot_sync(0xffffffffu, T > 0);
    int inc = T;
    for (int o = 1; o < p.B; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (range(__shfl_sync(0xffffffffu, inc, p.B - 1), __popc(some)))
      find(0, T, inc + w.slack * __popc(some & upto), 0);
    return w;
  }
  long long sum = 0;
  int n = 0;
#pragma unroll 4
  for (int b = lane; b < p.B; b += 32) {
    const int T = tree_tiles(p, b);
    sum += T;
    n += T > 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  if (!range(sum, n)) return w;
  long long before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const int T = b < p.B ? tree_tiles(p, b) : 0;
    long long inc = T > 0 ? T + w.slack : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (find(b0, T, inc, before)) break;
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return w;
}

// The next stretch of one unit's tiles in the range.
__device__ __forceinline__ bool tree_next(const TreeParams& p, TreeWalk& w, TreeSeg* s) {
  for (;;) {
    if (w.x >= w.hi) return false;
    while (w.x >= w.first + (long long)w.places() * p.Hkv) {
      w.first += (long long)w.places() * p.Hkv;
      if (++w.b >= p.B) return false;  // (the range ends at the list's end)
      w.T = tree_tiles(p, w.b);
    }
    const long long off = w.x - w.first;
    s->hkv = div_small(off, w.places());
    s->t0 = (int)(off - (long long)s->hkv * w.places());
    if (s->t0 < w.T) break;
    w.x += w.places() - s->t0;  // slack
  }
  s->b = w.b;
  s->T = w.T;
  s->L = tree_len(p, w.b);
  const long long left = w.hi - w.x;
  s->n = w.T - s->t0 < left ? w.T - s->t0 : (int)left;
  w.x += s->n;
  return true;
}

// The keys [0, at) and the tree's nodes `bits` from key `at` on, both relative
// to a tile.
__device__ __forceinline__ Mask128 tile_mask(int at, uint64_t bits) {
  Mask128 m{low_bits(at), low_bits(at - 64)};
  if (at <= -64 || at >= 128) return m;
  if (at < 0) {
    m.lo |= bits >> -at;
  } else if (at < 64) {
    m.lo |= bits << at;
    if (at > 0) m.hi |= bits >> (64 - at);
  } else {
    m.hi |= bits << (at - 64);
  }
  return m;
}
// Whole warp: ancestor masks of sequence b's nodes, lane l holding nodes l and
// l + 32, by pointer doubling (six rounds reach depth 64).  A node is unused
// when its parent entry is -2, is not a lower node (which also sets the bounds
// bit), or when its way up meets an unused node.  *used: the usable nodes.
__device__ __forceinline__ void tree_masks(const TreeParams& p, int b, uint64_t (&anc)[2],
                                           uint64_t* used) {
  const int lane = threadIdx.x & 31;
  int up[2];
  bool odd = false;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int s = lane + 32 * e;
    up[e] = -2;
    if (s < p.N) {
      const int v = p.parents[(size_t)b * p.N + s];
      up[e] = v >= -1 && v < s ? v : -2;
      odd |= v < -2 || v >= s;
    }
    anc[e] = 1ull << s;
  }
  if (odd) atomicOr(&g_tree_err, kErrBounds);
#pragma unroll
  for (int r = 0; r < 6; ++r) {
    uint64_t na[2];
    int nu[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = up[e] < 0 ? 0 : up[e];
      const uint64_t a0 = __shfl_sync(0xffffffffu, anc[0], t & 31);
      const uint64_t a1 = __shfl_sync(0xffffffffu, anc[1], t & 31);
      const int u0 = __shfl_sync(0xffffffffu, up[0], t & 31);
      const int u1 = __shfl_sync(0xffffffffu, up[1], t & 31);
      na[e] = up[e] < 0 ? anc[e] : anc[e] | (t < 32 ? a0 : a1);
      nu[e] = up[e] < 0 ? up[e] : (t < 32 ? u0 : u1);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      anc[e] = na[e];
      up[e] = nu[e];
    }
  }
  const uint64_t w0 = __ballot_sync(0xffffffffu, up[0] == -1);
  const uint64_t w1 = __ballot_sync(0xffffffffu, up[1] == -1);
  *used = w0 | w1 << 32;
}

template <int D, typename T, int MT>
__global__ void __launch_bounds__(tr::Cfg<D, MT>::THREADS, 1)
    tree_split_kernel(const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ TreeParams p) {
  using C = tr::Cfg<D, MT>;
  constexpr int NSTAGE = C::NSTAGE;
  constexpr int W_PROD = MT * 4, W_MMA = MT * 4 + 1;
  constexpr bool kBF16 = TileType<T>::kBF16;
  constexpr float NEG_INF = -INFINITY;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + C::SMEM_Q;
  uint64_t* full = reinterpret_cast<uint64_t*>(sKV + C::SMEM_KV);
  uint64_t* empty = full + NSTAGE;
  uint64_t* q_full = empty + NSTAGE;
  uint64_t* s_full = q_full + 1;  // [2] MT = 1: of alternate tiles; MT = 2: of the row tiles
  uint64_t* p_full = s_full + 2;  // [MT]
  uint64_t* pv_done = p_full + 2;  // [2] P V completed: MT = 1 of every tile, 2 of a stretch's last
  uint64_t* drain = pv_done + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile uint32_t* issued = reinterpret_cast<volatile uint32_t*>(abort_flag + 1);
  volatile uint32_t* tile_bad = issued + 1;  // [BAD_RING]
  static_assert(2 * C::NSTAGE * 8 + 8 * 8 + 12 + 4 * tr::BAD_RING <= C::SMEM_BAR, "barrier block");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x / p.n_rt, rt = blockIdx.x - group * p.n_rt;
  // Row tiles of this CTA that hold rows (the last CTA of a unit may have one).
  const int n_act = MT == 2 && p.rows - rt * C::RT > tr::BM ? 2 : 1;

  pdl_launch_dependents();
  if (threadIdx.x == W_PROD * 32) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, tr::BM * n_act);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], tr::BM);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *issued = 0;
    fence_mbar_init();
  }
  if (warp == W_MMA) {
    tmem_alloc(tmem_holder, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait_primary();  // everything below reads or writes the caller's memory

  TreeWalk w = tree_plan(p, group);
  TreeSeg sg = {};
  if (warp >= W_PROD) {
   if constexpr (MT == 2) regs_decrease<88>();
   if (warp == W_PROD) {
    // ============================ TMA producer ============================
    // Lane l < boxes * halves loads box l % boxes, half l / boxes of each tile.
    const int boxes = tr::BN / p.box;
    const int sub = lane % boxes, half = lane / boxes;
    const bool loads = half < C::HALVES;
    const uint64_t pol = p.n_rt == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
    uint32_t tc = 0;  // tiles so far: K at ring position 2 tc, V at 2 tc + 1
    bool ok = true;
    // Whole warp: ring position cnt may be overwritten.
    auto slot_free = [&](uint32_t cnt) {
      const uint32_t g = C::PAIRED ? (cnt + 1) >> 1 : cnt, n = C::PAIRED ? C::NPAIR : NSTAGE;
      return mbar_wait<true>(&empty[g % n], ((g / n) & 1) ^ 1, abort_flag, &g_tree_err, 1);
    };
    auto load = [&](uint32_t cnt, const CUtensorMap* m, uint64_t* bar, int id, int pos) {
      if (id >= 0)
        tma_load_4d_hint(
            sKV + (cnt % NSTAGE) * C::TILE_BYTES + half * tr::HALF_BYTES + sub * p.box * 128, m,
            bar, half * 64, sg.hkv, pos, id, pol);
    };
    auto tile_bytes = [&](int id) {
      return __popc(__ballot_sync(0xffffffffu, id >= 0)) * (uint32_t)p.box * 128u;
    };
    auto note_bad = [&](uint32_t t, int id) {
      const uint32_t bad = __ballot_sync(0xffffffffu, id == -2 && half == 0);
      if (lane == 0) {
        if (bad) atomicOr(&g_tree_err, kErrBounds);
        tile_bad[t % tr::BAD_RING] = bad;
      }
    };
    while (ok && tree_next(p, w, &sg)) {
      const int32_t* table = p.page_table + (size_t)sg.b * p.max_pages;
      // Page of this lane's box in tile t (-1: nothing to load, -2: no such
      // page) and the row in it.
      auto page_of = [&](int t, int* pos) {
        const int row = t * tr::BN + sub * p.box;
        if (!loads || row >= sg.L) return -1;
        const int pg = row / p.page_size;
        *pos = row - pg * p.page_size;
        const int id = table[pg];
        return id < 0 || id >= p.num_pages ? -2 : id;
      };
      // Ring order K_0, V_0, K_1, V_1, ...; pages are looked up two tiles ahead.
      int pos = 0, pos_n = 0, pos_nn = 0;
      int id = page_of(sg.t0, &pos), id_n = sg.n > 1 ? page_of(sg.t0 + 1, &pos_n) : -1;
      if (!(ok = slot_free(2 * tc))) break;
      {
        const uint32_t s = (2 * tc) % NSTAGE, bytes = tile_bytes(id);
        note_bad(tc, id);
        if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
        __syncwarp();
        load(2 * tc, &tmK, &full[s], id, pos);
        if (lane == 0) *issued = 2 * tc + 1;
      }
      for (int j = 0; j < sg.n && ok; ++j, ++tc) {
        const uint32_t cv = 2 * tc + 1, ck = cv + 1;
        const bool more = j + 1 < sg.n;
        const int id_nn = j + 2 < sg.n ? page_of(sg.t0 + j + 2, &pos_nn) : -1;
        const uint32_t vb = tile_bytes(id), kb = tile_bytes(id_n);
        if (!(ok = slot_free(cv))) break;
        if (C::PAIRED && more) {
          // V_j completes on K_{j+1}'s barrier; its own gets a plain arrival
          // that keeps its phases in step.
          note_bad(tc + 1, id_n);
          uint64_t* bar = &full[ck % NSTAGE];
          if (lane == 0) {
            mbar_arrive_expect_tx(bar, vb + kb);
            mbar_arrive(&full[cv % NSTAGE]);
          }
          __syncwarp();
          load(cv, &tmV, bar, id, pos);
          load(ck, &tmK, bar, id_n, pos_n);
        } else {
          if (lane == 0) mbar_arrive_expect_tx(&full[cv % NSTAGE], vb);
          __syncwarp();
          load(cv, &tmV, &full[cv % NSTAGE], id, pos);
          if (more) {
            if (lane == 0) *issued = cv + 1;
            if (!(ok = slot_free(ck))) break;
            note_bad(tc + 1, id_n);
            if (lane == 0) mbar_arrive_expect_tx(&full[ck % NSTAGE], kb);
            __syncwarp();
            load(ck, &tmK, &full[ck % NSTAGE], id_n, pos_n);
          }
        }
        if (lane == 0) *issued = more ? ck + 1 : cv + 1;
        id = id_n;
        pos = pos_n;
        id_n = id_nn;
        pos_n = pos_nn;
      }
    }
    __syncwarp();
    // The first CTA's producer, done early, lists where each sequence starts for
    // the merge.
    if (blockIdx.x == 0) {
      long long before = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int T = b0 + lane < p.B ? tree_tiles(p, b0 + lane) : 0;
        long long inc = T > 0 ? (long long)(T + w.slack) * p.Hkv : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        if (b0 + lane < p.B) {
          p.start[b0 + lane + 1] = before + inc;
          if ((long long)p.seqlens[b0 + lane] > (long long)p.max_pages * p.page_size)
            atomicOr(&g_tree_err, kErrBounds);
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) {
        p.start[0] = 0;
        p.start[p.B + 1] = w.slack;
      }
    }
   } else if (warp == W_MMA) {
    // ============================ MMA issuer (lane 0) ============================
    if (lane == 0) {
      constexpr uint32_t IDESC_S = idesc_f16(tr::BM, tr::BN, kBF16, false);
      constexpr uint32_t IDESC_O = idesc_f16(tr::BM, D, kBF16, true);
      const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dk = sdesc_sw128(smem_u32(sKV), 16, 1024);
      const uint64_t dv = sdesc_sw128(smem_u32(sKV), tr::HALF_BYTES, 1024);
      const uint32_t sd_hi = (uint32_t)(dq >> 32);
      const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, v_lo = (uint32_t)dv;
      // S[buf] = Q[tile] K^T, over D / 16 steps.
      auto issue_s = [&](int tile, int buf, uint32_t stage) {
        const uint32_t a0 = q_lo + tile * (C::TILE_BYTES >> 4);
        const uint32_t b0 = k_lo + stage * (C::TILE_BYTES >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * tr::HALF_BYTES + (k & 3) * 32) >> 4;
          mma_ss_lh(tmem + C::COL_S + buf * 128, a0 + off, sd_hi, b0 + off, sd_hi, IDESC_S,
                    k > 0 ? 1u : 0u);
        }
      };
      // O[tile] (+)= P[buf] V, over 128 / 16 steps.
      auto issue_pv = [&](int tile, int buf, uint32_t stage, bool add) {
        const uint32_t b0 = v_lo + stage * (C::TILE_BYTES >> 4);
#pragma unroll
        for (int k = 0; k < tr::BN / 16; ++k)
          mma_ts_lh(tmem + C::COL_O + tile * D, tmem + C::COL_S + buf * 128 + k * 8,
                    b0 + (uint32_t)((k * 16 * 128) >> 4), sd_hi, IDESC_O, add || k > 0 ? 1u : 0u);
      };
      uint32_t tc = 0, sc = 0;
      bool ok = true;
      auto landed = [&](uint32_t cnt, unsigned site) {
        const bool r = mbar_wait<false>(&full[cnt % NSTAGE], (cnt / NSTAGE) & 1, abort_flag,
                                       &g_tree_err, site);
        tc_fence_after();
        return r;
      };
      while (ok && tree_next(p, w, &sg)) {
        if (!(ok = mbar_wait<false>(q_full, sc & 1, abort_flag, &g_tree_err, 2))) break;
        ++sc;
        tc_fence_after();
        if (!(ok = landed(2 * tc, 3))) break;
        if constexpr (MT == 1) {
          issue_s(0, tc & 1, (2 * tc) % NSTAGE);
          mma_commit(&s_full[tc & 1]);
          mma_commit(&empty[(2 * tc) % NSTAGE]);
          for (int j = 0; j < sg.n; ++j, ++tc) {
            const uint32_t ck = 2 * tc + 2, cv = 2 * tc + 1;
            if (j + 1 < sg.n) {
              // S of the next tile goes ahead of this tile's P V, so that it is
              // ready when the softmax warps get to it.  (Its buffer held P of
              // the tile before this one, whose P V was issued earlier.)
              if (!(ok = landed(ck, 4))) break;
              issue_s(0, (tc + 1) & 1, ck % NSTAGE);
              mma_commit(&s_full[(tc + 1) & 1]);
              mma_commit(&empty[ck % NSTAGE]);
            }
            if (!(ok = landed(cv, 5))) break;
            if (!(ok = mbar_wait<false>(&p_full[0], tc & 1, abort_flag, &g_tree_err, 6))) break;
            tc_fence_after();
            issue_pv(0, tc & 1, cv % NSTAGE, j > 0);
            mma_commit(&pv_done[0]);
            mma_commit(&empty[cv % NSTAGE]);
          }
        } else {
          issue_s(0, 0, (2 * tc) % NSTAGE);
          mma_commit(&s_full[0]);
          if (n_act == 2) {
            issue_s(1, 1, (2 * tc) % NSTAGE);
            mma_commit(&s_full[1]);
          }
          // K_0 completes its pair with the stretch before's last V.
          mma_commit(&empty[tc % C::NPAIR]);
          for (int j = 0; j < sg.n; ++j, ++tc) {
            const uint32_t ck = 2 * tc + 2, cv = 2 * tc + 1;
            const bool more = j + 1 < sg.n;
            if (!(ok = landed(more ? ck : cv, 5))) break;
            if (!(ok = mbar_wait<false>(&p_full[0], tc & 1, abort_flag, &g_tree_err, 6))) break;
            tc_fence_after();
            issue_pv(0, 0, cv % NSTAGE, j > 0);
            if (more) {
              issue_s(0, 0, ck % NSTAGE);
              mma_commit(&s_full[0]);
            } else {
              mma_commit(&pv_done[0]);
            }
            if (n_act == 2) {
              if (!(ok = mbar_wait<false>(&p_full[1], tc & 1, abort_flag, &g_tree_err, 7))) break;
              tc_fence_after();
              issue_pv(1, 1, cv % NSTAGE, j > 0);
              if (more) {
                issue_s(1, 1, ck % NSTAGE);
                mma_commit(&s_full[1]);
              } else {
                mma_commit(&pv_done[1]);
              }
            }
            if (more) mma_commit(&empty[(tc + 1) % C::NPAIR]);
          }
        }
      }
      // Every MMA issued here has completed before tensor memory is freed.
      mma_commit(drain);
      mbar_wait_drain(drain, 0);
    }
    __syncwarp();
   }
  } else if ((warp >> 2) < n_act) {
    if constexpr (MT == 2) regs_increase<208>();
    // ======================= softmax and epilogue =======================
    const int i = warp >> 2, wq = warp & 3;
    const int tid = wq * 32 + lane;             // row within the tile, and V row it clears
    const int rr = i * tr::BM + tid;            // row within the CTA
    const int r = rt * C::RT + rr;              // row (s, g) of the kv head
    const bool row_ok = r < p.rows;
    const bool warp_ok = rt * C::RT + i * tr::BM + wq * 32 < p.rows;
    const int s = row_ok ? r / p.G : 0, g = row_ok ? r - s * p.G : 0;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t tO = t_lane + C::COL_O + i * D;
    const float c = p.c;
    const bool neg = c < 0.f;
    const float hide = neg ? -NEG_INF : NEG_INF;
    uint32_t tc = 0, seg = 0;
    int cur_b = -1;
    uint64_t anc = 0, used = 0;
    bool ok = true;
    // This row of Q for a stretch, in the swizzled layout of a TMA load.  Done
    // as soon as S of the stretch before's last tile is there (no MMA reads Q
    // any more), so that the next stretch's S runs under the epilogue.
    auto load_q = [&](const TreeSeg& t) {
      const T* const src = static_cast<const T*>(p.q) +
                           (((size_t)t.b * p.N + s) * p.Hq + (size_t)t.hkv * p.G + g) * D;
      put_q_row<D>(sQ + i * C::TILE_BYTES, tid, src, row_ok);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(q_full);
    };
    bool have = tree_next(p, w, &sg);
    if (have) load_q(sg);
    while (have) {
      if (sg.b != cur_b) {
        cur_b = sg.b;
        uint64_t a[2];
        tree_masks(p, cur_b, a, &used);
        const uint64_t a0 = __shfl_sync(0xffffffffu, a[0], s & 31);
        const uint64_t a1 = __shfl_sync(0xffffffffu, a[1], s & 31);
        anc = s < 32 ? a0 : a1;
      }
      const size_t qrow = ((size_t)sg.b * p.N + s) * p.Hq + (size_t)sg.hkv * p.G + g;
      const int base = sg.L - p.N;  // keys before the tree
      float m_used = NEG_INF, l = 0.f;
      for (int j = 0; j < sg.n; ++j, ++tc) {
        const int buf = MT == 1 ? tc & 1 : i;
        const uint32_t tS = t_lane + C::COL_S + buf * 128;
        const uint32_t par = MT == 1 ? (tc >> 1) & 1 : tc & 1;
        if (!(ok = mbar_wait<false>(&s_full[buf], par, abort_flag, &g_tree_err, 8 + i))) break;
        __syncwarp();
        tc_fence_after();
        const int kv0 = (sg.t0 + j) * tr::BN;
        const uint32_t bad = tile_bad[tc % tr::BAD_RING];
        const bool masked = kv0 > base - tr::BN || bad;
        if (masked) {
          // V rows that no query may see (unused nodes, slots past the end,
          // bad pages) can hold anything: they are cleared, since 0 * NaN in
          // P V would reach every row.
          const Mask128 any = tile_mask(base - kv0, used), fine = sound_keys(bad, p.box);
          const Mask128 keep{any.lo & fine.lo, any.hi & fine.hi};
          const uint32_t cv = 2 * tc + 1;
          const uint32_t on = C::PAIRED && j + 1 < sg.n ? cv + 1 : cv;  // V's barrier
          if (!(ok = mbar_wait<false>(&full[on % NSTAGE], (on / NSTAGE) & 1, abort_flag,
                                      &g_tree_err, 10)))
            break;
          clear_rows<D>(sKV + (cv % NSTAGE) * C::TILE_BYTES, wq, lane, keep);
        }
        // MT = 1: (the stretch before waited for its last P V.)  MT = 2: S of
        // this tile was issued after P V of the last, and both are done.
        bool pv_waited = MT == 2 || j == 0;
        if (warp_ok) {
          auto mask = [&](uint32_t (&sr)[4][32]) {
            const Mask128 fine = sound_keys(bad, p.box), mine = tile_mask(base - kv0, anc);
            hide_keys(sr, Mask128{mine.lo & fine.lo, mine.hi & fine.hi}, hide);
          };
          // O of the tiles so far may be rescaled once the last of their P V is done.
          auto settled = [&] {
            if (!pv_waited && !(ok = mbar_wait<false>(&pv_done[i], (tc - 1) & 1, abort_flag,
                                                      &g_tree_err, 11)))
              return false;
            __syncwarp();
            pv_waited = true;
            return true;
          };
          if (!softmax_tile<D, T>(tS, tO, c, j == 0, masked, mask, settled, &m_used, &l)) break;
        }
        // MT = 1: one phase of pv_done per tile, each waited for before the next P
        // is handed over: the parity waits never fall two phases behind.
        if (!pv_waited && !(ok = mbar_wait<false>(&pv_done[i], (tc - 1) & 1, abort_flag,
                                                  &g_tree_err, 13)))
          break;
        tc_fence_before();
        mbar_arrive(&p_full[i]);
      }
      if (!ok) break;
      TreeSeg next = {};
      have = tree_next(p, w, &next);
      if (have) load_q(next);
      if (!(ok = mbar_wait<false>(&pv_done[i], (MT == 1 ? tc - 1 : seg) & 1, abort_flag,
                                  &g_tree_err, 15)))
        break;
      ++seg;
      __syncwarp();
      tc_fence_after();
      if (warp_ok) {
        // A row of an unused node gives O = 0 and log-sum-exp -inf.
        const bool live = used >> s & 1;
        if (!live) {
          l = 0.f;
          m_used = NEG_INF;
        }
        const bool whole = sg.t0 == 0 && sg.n == sg.T;
        const size_t part = (size_t)blockIdx.x * 2 + (sg.t0 > 0 ? 0 : 1);
        const size_t tile0 = part * (D / 4) * p.rt_rows + rr;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        if (row_ok) {
          if (whole) {
            // (A row with a score that is NaN has a sum and a log-sum-exp that are.)
            if (p.lse) p.lse[qrow] = l == 0.f ? NEG_INF : 0.6931471805599453f * (m_used + log2f(l));
          } else {
            reinterpret_cast<float2*>(p.part_ml)[part * p.rt_rows + rr] = make_float2(m_used, l);
          }
        }
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(tO + q * 32, o);
          tmem_wait_ld();
          reg_fence32(o);
          if (!row_ok) continue;
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.o) + qrow * D + q * 32);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t k[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float e0 = __uint_as_float(o[8 * x + 2 * y]) * inv;
                const float e1 = __uint_as_float(o[8 * x + 2 * y + 1]) * inv;
                k[y] = live ? TileType<T>::pack(e0, e1) : 0u;
              }
              dst[x] = make_uint4(k[0], k[1], k[2], k[3]);
            }
          } else {
            // [column / 4][row] of 16 bytes: the lanes' rows side by side.
            float4* dst = reinterpret_cast<float4*>(p.part_o) + tile0 + (size_t)q * 8 * p.rt_rows;
#pragma unroll
            for (int x = 0; x < 8; ++x)
              dst[(size_t)x * p.rt_rows] =
                  live ? make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                                     __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
      }
      tc_fence_before();
      sg = next;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  // After an abort: every load that may still be in flight, before the CTA
  // and its shared memory go.
  if (warp == W_PROD && *abort_flag) {
    const uint32_t n = *issued;
    for (uint32_t u = n > (uint32_t)NSTAGE ? n - NSTAGE : 0u; u < n; ++u)
      mbar_wait_drain(&full[u % NSTAGE], (u / NSTAGE) & 1);
    __syncwarp();
  }
}

// Merge of the units that several groups share, and zeros for padding
// sequences.  A thread takes 16 columns of a row, the lanes of a warp 32 rows of
// one (sequence, kv head), so that loads are as wide as the split kernel's
// stores; the partials' loads run kMergeAhead partials ahead, merged online
// (running max M, output and sum rescaled when it grows).
// KS = 1: a thread walks all of its row's partials.  KS = 8: the block's 8 warps
// share one set of 32 rows x 16 columns, each every 8th partial: with few rows
// a long cache leaves each of them up to one partial per SM.
constexpr int kMergeWarps = 8;
template <int D, typename T, int KS>
__global__ void __launch_bounds__(kMergeWarps * 32)
    tree_merge_kernel(const __grid_constant__ TreeParams p, int rt_size) {
  pdl_launch_dependents();
  pdl_wait_primary();
  constexpr int NC = D / 16;  // column chunks of a row
  constexpr int kMergeAhead = KS > 1 ? 4 : 2;
  __shared__ float sM[KS > 1 ? KS : 1][32], sDen[KS > 1 ? KS : 1][32];
  __shared__ float sAcc[KS > 1 ? KS : 1][16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Blocks of 32-row sets: KS = 1 takes 8 / NC sets, KS = 8 a chunk of one.
  const int sets = (p.rows + 31) / 32;
  int unit, set, chunk;
  if constexpr (KS == 1) {
    const int x = blockIdx.x * (kMergeWarps / NC) + warp / NC;
    unit = x / sets;
    set = x - unit * sets;
    chunk = warp % NC;
    if (unit >= p.B * p.Hkv) return;
  } else {
    const int x = blockIdx.x / NC;
    unit = x / sets;
    set = x - unit * sets;
    chunk = blockIdx.x - x * NC;
  }
  const int b = unit / p.Hkv, hkv = unit - b * p.Hkv;
  const long long first = p.start[b], after = p.start[b + 1], total = p.start[p.B];
  const int places = div_small(after - first, p.Hkv);
  int g0 = 0, g1 = -1;  // groups of the unit's tiles
  if (places > 0) {
    const long long u0 = first + (long long)hkv * places;
    const long long u1 = u0 + places - p.start[p.B + 1] - 1;
    // Group of place t: the largest g with total * g / G <= t.
    const long long G = tree_groups(p, total);
    g0 = (int)((u0 + 1) * G > 0xffffffffll ? ((u0 + 1) * G - 1) / total
                                           : (uint32_t)((u0 + 1) * G - 1) / (uint32_t)total);
    g1 = (int)((u1 + 1) * G > 0xffffffffll ? ((u1 + 1) * G - 1) / total
                                           : (uint32_t)((u1 + 1) * G - 1) / (uint32_t)total);
    if (g0 == g1) return;  // finished in place
  }
  const int r = set * 32 + lane;
  const bool real = r < p.rows;
  const int rt = real ? r / rt_size : 0, rr = real ? r - rt * rt_size : 0;
  float M = -INFINITY, den = 0.f, acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  auto scale = [&](float m) {  // the weight of values against max m
    if (m > M) {
      const float f = M == -INFINITY ? 0.f : fast_exp2(M - m);
      den *= f;
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] *= f;
      M = m;
    }
    return m == -INFINITY ? 0.f : fast_exp2(m - M);
  };
  float2 ml[kMergeAhead];
  float4 ov[kMergeAhead][4];
  auto load = [&](int k, int u) {
    ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) ov[u][e] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k <= g1 && real) {
      const size_t part = ((size_t)k * p.n_rt + rt) * 2 + (k == g0 ? 1 : 0);
      ml[u] = reinterpret_cast<const float2*>(p.part_ml)[part * p.rt_rows + rr];
      const float4* src = reinterpret_cast<const float4*>(p.part_o) +
                          (part * (D / 4) + chunk * 4) * p.rt_rows + rr;
#pragma unroll
      for (int e = 0; e < 4; ++e) ov[u][e] = src[(size_t)e * p.rt_rows];
    }
  };
  const int k0 = g0 + (KS > 1 ? warp : 0);
#pragma unroll
  for (int u = 0; u < kMergeAhead; ++u) load(k0 + u * KS, u);
  for (int k = k0; k <= g1; k += kMergeAhead * KS) {
#pragma unroll
    for (int u = 0; u < kMergeAhead; ++u) {
      const float wt = scale(ml[u].y > 0.f ? ml[u].x : -INFINITY);
      den += wt * ml[u].y;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[4 * e] += wt * ov[u][e].x;
        acc[4 * e + 1] += wt * ov[u][e].y;
        acc[4 * e + 2] += wt * ov[u][e].z;
        acc[4 * e + 3] += wt * ov[u][e].w;
      }
      load(k + (kMergeAhead + u) * KS, u);
    }
  }
  const int s = real ? r / p.G : 0;
  const size_t row = ((size_t)b * p.N + s) * p.Hq + (size_t)hkv * p.G + (r - s * p.G);
  T* const dst = static_cast<T*>(p.o) + row * D + chunk * 16;
  if constexpr (KS > 1) {
    // The warps' results meet in shared memory; then each warp finishes two of
    // the 16 columns.
    sM[warp][lane] = M;
    sDen[warp][lane] = den;
#pragma unroll
    for (int e = 0; e < 16; ++e) sAcc[warp][e][lane] = acc[e];
    __syncthreads();
    static_assert(KS == kMergeWarps && 2 * KS == 16, "two columns per warp");
    float m[KS];
    M = -INFINITY;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      m[i] = sM[i][lane];
      M = fmaxf(M, m[i]);
    }
    float a0 = 0.f, a1 = 0.f;
    den = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const float wt = m[i] == -INFINITY ? 0.f : fast_exp2(m[i] - M);
      den += wt * sDen[i][lane];
      a0 += wt * sAcc[i][2 * warp][lane];
      a1 += wt * sAcc[i][2 * warp + 1][lane];
    }
    if (!real) return;
    const float inv = den > 0.f ? 1.f / den : 0.f;
    reinterpret_cast<uint32_t*>(dst)[warp] = TileType<T>::pack(a0 * inv, a1 * inv);
    if (warp != 0) return;
  } else {
    if (!real) return;
    const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      reinterpret_cast<uint4*>(dst)[e] =
          make_uint4(TileType<T>::pack(acc[8 * e] * inv, acc[8 * e + 1] * inv),
                     TileType<T>::pack(acc[8 * e + 2] * inv, acc[8 * e + 3] * inv),
                     TileType<T>::pack(acc[8 * e + 4] * inv, acc[8 * e + 5] * inv),
                     TileType<T>::pack(acc[8 * e + 6] * inv, acc[8 * e + 7] * inv));
  }
  if (p.lse && chunk == 0)
    p.lse[row] = den == 0.f ? -INFINITY : 0.6931471805599453f * (M + log2f(den));
}

// Row tiles per CTA, row-tile CTAs per unit, tile groups.
struct TreePlan {
  int mt, n_rt, groups, rt_rows;
  size_t o_floats, ml_floats, bytes;
};
static TreePlan tree_host_plan(int B, int N, int Hq, int Hkv, long long cap, int D) {
  TreePlan t;
  // One row tile per CTA up to 128 rows, and where two would leave the last CTA of
  // a few half empty (D = 128, 336 rows: 68.5 us, with two 74.0; 600 rows 75.6 and
  // 80.0); else two (192 rows: 73.3 us, with one 82.3; 512 rows 68.2 and 75.3).
  const int rows = N * (Hq / Hkv), tiles = (rows + tr::BM - 1) / tr::BM;
  t.mt = tiles <= 5 && tiles % 2 == 1 ? 1 : 2;
  const int rt = t.mt * tr::BM;
  t.n_rt = (rows + rt - 1) / rt;
  t.rt_rows = rows < rt ? rows : rt;
  const int sms = sm_count() > 0 ? sm_count() : 148;
  long long g = sms / t.n_rt;
  const long long most = (long long)B * Hkv * ((cap + tr::BN - 1) / tr::BN);
  if (g > most) g = most;
  if (g < 1) g = 1;
  t.groups = (int)g;
  const size_t slots = (size_t)t.groups * t.n_rt * 2 * t.rt_rows;
  t.o_floats = slots * D;
  t.ml_floats = slots * 2;
  t.bytes = (t.o_floats + t.ml_floats) * sizeof(float) + ((size_t)B + 6) * sizeof(long long);
  return t;
}

template <int D, typename T, int MT>
static int launch_tree_t(const TreeParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                         cudaStream_t stream) {
  using C = tr::Cfg<D, MT>;
  static int attr_set[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE)) {
    e = cudaFuncSetAttribute(tree_split_kernel<D, T, MT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_TOTAL);
    if (e != cudaSuccess) return e;
    // The merge keeps the split kernel's division of the SM into L1 and shared
    // memory.  (Beside a split block there is no room for a merge block, in shared
    // memory or, for MT = 2, in registers.)  4 sequences of 16000 tokens, 128 rows per
    // kv head: 25.9 us so, 26.6 with the division left to the driver; 16 sequences
    // of up to 16384, 256 rows, 134.7 and 135.2; one of 2733, 32 rows, 11.2 and 11.05.
    for (auto k : {tree_merge_kernel<D, T, 1>, tree_merge_kernel<D, T, kMergeWarps>}) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout,
                               (int)cudaSharedmemCarveoutMaxShared);
      if (e != cudaSuccess) return e;
    }
    if (dev >= 0 && dev < 64) __atomic_store_n(&attr_set[dev], 1, __ATOMIC_RELEASE);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.groups * p.n_rt), 1, 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_TOTAL;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tree_split_kernel<D, T, MT>, tk, tv, p);
  if (e != cudaSuccess) return e;
  constexpr int NC = D / 16;
  const long long sets = (long long)p.B * p.Hkv * ((p.rows + 31) / 32);
  // Both kernels together, KS = 1 / 8: 64 rows of 22 partials 16.6 / 11.8 us, 512
  // rows of 5 partials 38.3 / 36.8 us, 2048 rows of 19 partials 68.4 / 64.1 us;
  // 8192 rows of 5 partials 189.6 / 198.7 us, 32768 rows of 2 140.9 / 174.7 us.
  const bool split = sets * NC <= 4 * (sm_count() > 0 ? sm_count() : 148);
  cfg.gridDim = dim3((unsigned)(split ? sets * NC : (sets * NC + kMergeWarps - 1) / kMergeWarps));
  cfg.blockDim = dim3(kMergeWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return split ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, T, kMergeWarps>, p, (int)C::RT)
               : cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, T, 1>, p, (int)C::RT);
}

template <int D, typename T>
static int launch_tree_d(const TreeParams& p, int mt, const CUtensorMap& tk, const CUtensorMap& tv,
                         cudaStream_t stream) {
  return mt == 1 ? launch_tree_t<D, T, 1>(p, tk, tv, stream)
                 : launch_tree_t<D, T, 2>(p, tk, tv, stream);
}

// A cache without capacity: every row is a padding sequence's, and any token is
// past the page table.
__global__ void tree_zero_kernel(uint16_t* o, size_t n, float* lse, size_t nl,
                                 const int32_t* seqlens, size_t B) {
  const size_t at = blockIdx.x * (size_t)blockDim.x + threadIdx.x;
  const size_t step = (size_t)gridDim.x * blockDim.x;
  for (size_t i = at; i < n; i += step) o[i] = 0;
  if (lse)
    for (size_t i = at; i < nl; i += step) lse[i] = -INFINITY;
  bool past = false;
  for (size_t i = at; i < B; i += step) past |= seqlens[i] > 0;
  if (past) atomicOr(&g_tree_err, kErrBounds);
}

int set_tree_wait_limit(unsigned long long ns) { return set_wait_limit_this_unit(ns); }

int read_tree_error(unsigned int* out, int reset) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_tree_err, sizeof(v));
  if (e != cudaSuccess) return e;
  if (reset && v) {
    const unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_tree_err, &z, sizeof(z));
    if (e != cudaSuccess) return e;
  }
  *out = v;
  return cudaSuccess;
}

}  // namespace fa

static bool al(const void* p, unsigned n) {
  return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

extern "C" int fa_decode_tree_fwd(const void* q, const void* kpages, const void* vpages,
                                  const int32_t* page_table, const int32_t* seqlens,
                                  const int32_t* parents, void* o, float* lse, int B, int N,
                                  int Hq, int Hkv, int num_pages, int page_size, int max_pages,
                                  int D, float scale, int dtype, cudaStream_t stream) {
  if (B < 0 || N < 0 || Hq < 0 || Hkv < 0 || num_pages < 0 || max_pages < 0)
    return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_INVALID_ARG;
  if (!isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (page_size < 32 || page_size % 32 != 0) return FA_ERR_INVALID_ARG;
  if (N > fa::tr::MAX_N) return FA_ERR_UNSUPPORTED;
  if (B == 0 || N == 0 || Hq == 0) return FA_OK;
  if (Hkv == 0 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  // Row indexes and the merge's grid (at most one block per row) fit 31 bits.
  if ((int64_t)B * N * Hq > INT32_MAX) return FA_ERR_INVALID_ARG;
  if ((int64_t)max_pages * page_size > INT32_MAX) return FA_ERR_INVALID_ARG;
  if (!al(q, 16) || !al(o, 16)) return FA_ERR_INVALID_ARG;
  if (lse && !al(lse, 4)) return FA_ERR_INVALID_ARG;
  if (!al(seqlens, 4)) return FA_ERR_INVALID_ARG;
  if (max_pages > 0 && (num_pages < 1 || !al(kpages, 16) || !al(vpages, 16) ||
                        !al(page_table, 4) || !al(parents, 4)))
    return FA_ERR_INVALID_ARG;
  if ((int64_t)num_pages * page_size > (1ll << 40) / (2 * D) / Hkv) return FA_ERR_INVALID_ARG;
  const fa::SetupDuringCapture setup;
  if (max_pages == 0) {
    const size_t rows = (size_t)B * N * Hq, n = rows * D;
    fa::tree_zero_kernel<<<(unsigned)((n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096), 256, 0,
                           stream>>>(static_cast<uint16_t*>(o), n, lse, rows, seqlens, (size_t)B);
    return fa::record_cuda_status(cudaGetLastError(), "tree decode zero-fill launch");
  }
  const fa::TreePlan t =
      fa::tree_host_plan(B, N, Hq, Hkv, (long long)max_pages * page_size, D);
  fa::TreeParams p = {};
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.page_table = page_table;
  p.seqlens = seqlens;
  p.parents = parents;
  p.B = B;
  p.N = N;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.rows = N * p.G;
  p.rt_rows = t.rt_rows;
  p.n_rt = t.n_rt;
  p.groups = t.groups;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  // Keys per TMA box: a tile's boxes must not straddle pages.
  p.box = page_size % 128 == 0 ? 128 : (page_size % 64 == 0 ? 64 : 32);
  p.c = scale * 1.4426950408889634f;
  // scale == 0: every visible score is 0; a tiny c keeps hidden keys at -inf.
  if (p.c == 0.f) p.c = 1e-30f;
  CUtensorMap tk, tv;
  if (fa::encode_tmap_rows(&tk, kpages, D, Hkv, page_size, num_pages, p.box) ||
      fa::encode_tmap_rows(&tv, vpages, D, Hkv, page_size, num_pages, p.box))
    return fa::record_cuda_status(cudaErrorInvalidValue, "tree decode tensor maps");
  void* scratch = nullptr;
  cudaError_t e = fa::scratch_alloc(&scratch, t.bytes, stream);
  if (e != cudaSuccess) return fa::record_cuda_status(e, "tree decode scratch");
  p.start = static_cast<long long*>(scratch);
  // (B + 2) 8-byte entries, then the partials 32-byte aligned.
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) +
                                      (((size_t)B + 2) * 8 + 31) / 32 * 32);
  p.part_ml = p.part_o + t.o_floats;
  int r;
  const bool bf16 = dtype == FA_BF16;
  if (D == 64)
    r = bf16 ? fa::launch_tree_d<64, __nv_bfloat16>(p, t.mt, tk, tv, stream)
             : fa::launch_tree_d<64, __half>(p, t.mt, tk, tv, stream);
  else
    r = bf16 ? fa::launch_tree_d<128, __nv_bfloat16>(p, t.mt, tk, tv, stream)
             : fa::launch_tree_d<128, __half>(p, t.mt, tk, tv, stream);
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  if (r != 0) return fa::record_cuda_status(r, "tree decode launch");
  return fa::record_cuda_status(ef, "tree decode cudaFreeAsync");
}
