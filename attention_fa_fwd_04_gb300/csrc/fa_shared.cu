// fa_shared.cu -- attention of new tokens over a paged cache whose sequences share
// long prefixes (fa_decode_shared_fwd).
//
// What it computes: fa_decode_paged_fwd's rows.  Query row (b, s, h) attends to the
// keys [0, L_b - Sq + s]; the first P_g of them, those of its group's prefix, lie in
// the same pages for the whole group.
//   O = sum_j p_j V_j / sum_j p_j,  p_j = exp(scale <q, K_j> - max)
// splits by keys: with partial results (m, l, O) of the prefix and of the
// sequence's own keys, weights 2^(m - max) join them.
//
// Floor: each prefix's K/V once and each sequence's own K/V once from HBM, and
// 4 D operations per (row, key).  All rows of a group (members x Sq x G per kv
// head) meet each prefix tile, so from about 256 rows on the matrix units bound
// the prefix, below that the cache stream; own keys are always bound by the stream.
//
// Design: every (group, kv head) and every (sequence, kv head) is a unit of rows
// against a range of 128-key tiles, done by tcgen05 MMAs as in the tree decode (S
// and O in tensor memory, P written back over S).  A CTA has two softmax
// warpgroups, one TMA producer warp and one MMA warp.  Units of more than 128 rows
// give each warpgroup a 128-row tile, and both meet every key tile; with fewer rows
// the warpgroups take alternate key tiles of the one row tile, each with sums of its
// own, so that the softmax of one runs beside the other's.
// Split: lengths, prefixes and groups are device data.  The tiles of all units form
// one list, cut into equal ranges, one per CTA.  A unit of several row-tile pairs is
// cut into strips of keys about as long as a range, and the pairs of one strip stand
// side by side in the list, so that the CTAs which read the same keys do so at the
// same time and share them through L2.  Every stretch of a range leaves a partial; a
// second kernel merges a row's.
#include <math.h>

#include <type_traits>

#include "fa.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_tiles.cuh"

namespace fa {

__device__ unsigned int g_shared_err = 0;

namespace sh {
using namespace tiles;
constexpr int MAX_GROUPS = 1024;  // their starts lie in shared memory
constexpr int THREADS = 384;
constexpr int WARPS = THREADS / 32;
constexpr int SLACK = 4;  // places without a tile after each stretch, for what it costs beside

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE_BYTES = HALVES * HALF_BYTES;
  static constexpr int NSTAGE = D == 128 ? 4 : 10;  // K and V tiles in flight
  static constexpr int SMEM_Q = 2 * TILE_BYTES;
  static constexpr int SMEM_KV = NSTAGE * TILE_BYTES;
  static constexpr int SMEM_BAR = 512, SMEM_PLAN = 256;
  static constexpr int SMEM_STARTS = (MAX_GROUPS + 4) * 4;
  static constexpr int SMEM_TOTAL = 1024 + SMEM_Q + SMEM_KV + SMEM_BAR + SMEM_PLAN + SMEM_STARTS;
  static_assert(SMEM_TOTAL <= 227 * 1024, "shared memory per CTA");
  static_assert(NSTAGE / 2 + 2 < BAD_RING, "tiles in flight");
  // Tensor memory: S of each warpgroup, then O of each.
  static constexpr uint32_t COL_S = 0, COL_O = 256, TMEM_COLS = 512;
};
}  // namespace sh

struct SharedParams {
  const void* q;  // [B, Sq, Hq, D]
  void* o;
  float* lse;  // [B, Sq, Hq] or null
  const int32_t* page_table;
  const int32_t* seqlens;
  const int32_t* starts;  // [groups + 1]
  const int32_t* prefix;  // [groups]
  // Partials of group units and of sequence units: [id][D / 4][2 * half][4]
  // unnormalised outputs, [id][2 * half][2] (max in log2 units, sum).
  float* part_o[2];
  float* part_ml[2];
  int half[2];         // rows of a warpgroup in a slot
  long long* first;    // [owners + 1] first place of each owner, then strip width, slack
  int* pieces;         // [owners] pieces of the owners of its kind before it
  int B, groups, Sq, Hq, Hkv, G, SqG;
  int page_size, max_pages, num_pages, box, ctas;
  float c;  // scale * log2(e)
};

// a / b in 32 bits where both fit.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Owners of units: group g is owner g, sequence b owner groups + b.
struct Shape {
  int rows;        // query rows per kv head
  int row0;        // first sequence
  int tab;         // sequence whose row of the page table lists the keys
  int lo, hi;      // keys [lo, hi)
  int t0, T;       // first tile and tiles
  int n_rt;        // pairs of row tiles
  int S, len;      // strips, tiles of each but the last
};
__device__ __forceinline__ long long places_per_head(const Shape& s, int slack) {
  return (long long)s.n_rt * (s.T + (long long)s.S * slack);
}
__device__ __forceinline__ long long shared_cap(const SharedParams& p) {
  return (long long)p.max_pages * p.page_size;
}
__device__ __forceinline__ int shared_len(const SharedParams& p, int b) {
  const int L = p.seqlens[b];
  return L < 0 ? 0 : (L > shared_cap(p) ? (int)shared_cap(p) : L);
}
// Tokens that group g shares: 0 for fewer than two members.
__device__ __forceinline__ int group_prefix(const SharedParams& p, const int* starts, int g) {
  if (starts[g + 1] - starts[g] < 2) return 0;
  const int P = p.prefix[g];
  return P < 0 || P > shared_cap(p) ? 0 : P;
}
// The group of sequence b, or -1.  groups: 0 where the starts are not sound.
__device__ __forceinline__ int group_of(const int* starts, int groups, int b) {
  if (groups == 0 || b < starts[0] || b >= starts[groups]) return -1;
  int lo = 0, hi = groups;  // starts[lo] <= b < starts[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= b)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}
// Keys of sequence b that its group's unit covers: all of the prefix, or none for a
// sequence that is not past it.
__device__ __forceinline__ int covered(const SharedParams& p, const int* starts, int groups,
                                       int b, int L) {
  const int g = group_of(starts, groups, b);
  if (g < 0) return 0;
  const int P = group_prefix(p, starts, g);
  return L - p.Sq + 1 >= P ? P : 0;
}
// W: tiles of a CTA's range, 0 while it is not known.
__device__ __forceinline__ Shape shape_of(const SharedParams& p, const int* starts, int groups,
                                          int o, int W) {
  Shape s;
  if (o < p.groups) {
    const bool real = o < groups;
    s.lo = 0;
    s.hi = real ? group_prefix(p, starts, o) : 0;
    s.row0 = real ? starts[o] : 0;
    s.rows = real ? (starts[o + 1] - starts[o]) * p.SqG : 0;
    // The first member that is past the prefix; without one there is nothing to do.
    s.tab = s.row0;
    if (s.hi > 0) {
      while (s.tab < starts[o + 1] && shared_len(p, s.tab) - p.Sq + 1 < s.hi) ++s.tab;
      if (s.tab == starts[o + 1]) s.hi = 0;
    }
  } else {
    const int b = o - p.groups, L = shared_len(p, b);
    s.row0 = s.tab = b;
    s.rows = p.SqG;
    s.hi = L;
    s.lo = covered(p, starts, groups, b, L);
  }
  s.t0 = s.lo / sh::BN;
  s.T = s.hi > s.lo ? (int)(((uint32_t)s.hi + sh::BN - 1) / sh::BN) - s.t0 : 0;
  s.n_rt = (s.rows + 2 * sh::BM - 1) / (2 * sh::BM);
  s.S = W > 0 ? max(1, s.T / W) : 1;
  s.len = (s.T + s.S - 1) / s.S;
  s.S = s.len > 0 ? (s.T + s.len - 1) / s.len : 1;
  return s;
}

// A CTA's place in the list.
struct SharedWalk {
  long long x, hi;  // next and last place of the range
  long long first;  // first place of owner o
  int o, piece0;    // owner; pieces of its kind before it
  int W, slack, groups;
  Shape s;
};
struct SharedSeg {
  int kind;  // 0 group, 1 sequence
  int hkv, rt, t, n, id;
};

__device__ __forceinline__ bool shared_next(const SharedParams& p, const int* starts,
                                            SharedWalk& w, SharedSeg* g) {
  int s, rt, at, len;
  for (;;) {
    if (w.x >= w.hi) return false;
    long long per = places_per_head(w.s, w.slack);
    while (w.x >= w.first + per * p.Hkv || w.s.T == 0) {
      if (w.s.T > 0) {
        w.first += per * p.Hkv;
        w.piece0 += p.Hkv * w.s.S * w.s.n_rt;
      }
      if (++w.o >= p.groups + p.B) return false;  // (the range ends at the list's end)
      if (w.o == p.groups) w.piece0 = 0;
      w.s = shape_of(p, starts, w.groups, w.o, w.W);
      per = places_per_head(w.s, w.slack);
    }
    long long y = w.x - w.first;
    g->hkv = (int)quotient(y, per);
    y -= g->hkv * per;
    const long long strip = (long long)w.s.n_rt * (w.s.len + w.slack);
    s = (int)quotient(y, strip);
    const long long z = y - s * strip;
    len = min(w.s.len, w.s.T - s * w.s.len);
    rt = (int)quotient(z, len + w.slack);
    at = (int)(z - (long long)rt * (len + w.slack));
    if (at < len) break;
    w.x += len + w.slack - at;  // slack
  }
  const long long left = w.hi - w.x;
  g->kind = w.o < p.groups ? 0 : 1;
  g->rt = rt;
  g->t = w.s.t0 + s * w.s.len + at;
  g->n = len - at < left ? len - at : (int)left;
  // Stretches in list order: each begins a piece or a CTA's range.
  g->id = w.piece0 + (g->hkv * w.s.S + s) * w.s.n_rt + rt + (int)blockIdx.x;
  w.x += g->n;
  return true;
}

// Query row r of a unit: its index in [B, Sq, Hq].
__device__ __forceinline__ size_t shared_qrow(const SharedParams& p, int row0, int hkv, int r,
                                              int* s_out) {
  const int m = r / p.SqG, e = r - m * p.SqG, s = e / p.G;
  *s_out = s;
  return ((size_t)(row0 + m) * p.Sq + s) * p.Hq + (size_t)hkv * p.G + (e - s * p.G);
}

// Block-wide: the list, and this CTA's range of it.  starts: shared memory for the
// groups' starts; plan: shared scratch.  CTA 0 also writes it down for the merge.
struct PlanScratch {
  long long sums[2 * sh::WARPS];
  long long first;
  int o, piece0, sound;
};
__device__ __forceinline__ SharedWalk shared_plan(const SharedParams& p, int* starts,
                                                  PlanScratch* sc) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int owners = p.groups + p.B;
  if (t == 0) {
    sc->sound = 1;
    sc->o = -1;
  }
  for (int i = t; i <= p.groups && p.groups > 0; i += sh::THREADS) starts[i] = p.starts[i];
  __syncthreads();
  if (p.groups > 0) {
    bool odd = false, far = false;
    for (int i = t; i <= p.groups; i += sh::THREADS) {
      odd |= starts[i] < 0 || starts[i] > p.B || (i > 0 && starts[i] < starts[i - 1]);
      if (blockIdx.x == 0 && i < p.groups) far |= p.prefix[i] < 0 || p.prefix[i] > shared_cap(p);
    }
    if (odd) sc->sound = 0;
    if ((odd && blockIdx.x == 0) || far) atomicOr(&g_shared_err, kErrBounds);
    __syncthreads();
  }
  SharedWalk w;
  w.groups = sc->sound ? p.groups : 0;
  // Inclusive sums over the block, and totals.
  auto scan = [&](long long& a, long long& b, long long* ta, long long* tb) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
      if (lane >= o) {
        a += x;
        b += y;
      }
    }
    __syncthreads();
    if (lane == 31) {
      sc->sums[2 * warp] = a;
      sc->sums[2 * warp + 1] = b;
    }
    __syncthreads();
    *ta = *tb = 0;
    for (int i = 0; i < sh::WARPS; ++i) {
      if (i == warp) {
        a += *ta;
        b += *tb;
      }
      *ta += sc->sums[2 * i];
      *tb += sc->sums[2 * i + 1];
    }
  };
  long long raw = 0, total = 0, unused;
  Shape mine;  // of this thread's first owner
  for (int o = t; o < owners; o += sh::THREADS) {
    const Shape s = shape_of(p, starts, w.groups, o, 0);
    if (o == t) mine = s;
    raw += (long long)p.Hkv * s.n_rt * s.T;
  }
  long long zero = 0, sum;
  scan(raw, zero, &sum, &unused);
  const long long n = p.ctas;
  const long long width = quotient(sum + n - 1, n);
  w.W = width < 1 ? 1 : (width > INT32_MAX ? INT32_MAX : (int)width);
  w.slack = sum > n ? sh::SLACK : 0;
  auto strips = [&](Shape s) {
    s.S = max(1, s.T / w.W);
    s.len = (s.T + s.S - 1) / s.S;
    s.S = s.len > 0 ? (s.T + s.len - 1) / s.len : 1;
    return s;
  };
  for (int o = t; o < owners; o += sh::THREADS) {
    const Shape s = strips(o == t ? mine : shape_of(p, starts, w.groups, o, 0));
    if (s.T > 0) total += p.Hkv * places_per_head(s, w.slack);
  }
  zero = 0;
  scan(total, zero, &sum, &unused);
  const long long used = sum < n ? sum : n, c = blockIdx.x;
  w.x = c < used ? mul_div(sum, (int)c, used) : 0;
  w.hi = c < used ? mul_div(sum, (int)c + 1, used) : 0;
  if (c >= used && c > 0) return w;  // (block-uniform)
  long long places0 = 0, pieces0 = 0;  // pieces: groups' in the upper half, sequences' in the lower
  for (int o0 = 0; o0 < owners; o0 += sh::THREADS) {
    const int o = o0 + t;
    long long places = 0, pieces = 0, my_places = 0, my_pieces = 0, all_places, all_pieces;
    if (o < owners) {
      const Shape s = strips(o == t ? mine : shape_of(p, starts, w.groups, o, 0));
      if (s.T > 0) {
        my_places = p.Hkv * places_per_head(s, w.slack);
        my_pieces = (long long)p.Hkv * s.S * s.n_rt;
        if (o < p.groups) my_pieces <<= 32;
      }
    }
    places = my_places;
    pieces = my_pieces;
    scan(places, pieces, &all_places, &all_pieces);
    const long long first = places0 + places - my_places, before = pieces0 + pieces - my_pieces;
    const int piece0 = o < p.groups ? (int)(before >> 32) : (int)before;
    if (o < owners) {
      if (my_places > 0 && first <= w.x && w.x < first + my_places && w.x < w.hi) {
        sc->o = o;
        sc->first = first;
        sc->piece0 = piece0;
      }
      if (blockIdx.x == 0) {
        p.first[o] = first;
        p.pieces[o] = piece0;
      }
    }
    places0 += all_places;
    pieces0 += all_pieces;
    if (blockIdx.x != 0 && places0 > w.x) break;  // (block-uniform)
  }
  if (blockIdx.x == 0 && t == 0) {
    p.first[owners] = places0;
    p.first[owners + 1] = w.W;
    p.first[owners + 2] = w.slack;
    p.first[owners + 3] = w.groups;
  }
  __syncthreads();
  w.o = sc->o;
  w.first = sc->first;
  w.piece0 = sc->piece0;
  if (w.o < 0) {
    w.hi = w.x;
    return w;
  }
  w.s = shape_of(p, starts, w.groups, w.o, w.W);
  return w;
}

template <int D, typename T>
__global__ void __launch_bounds__(sh::THREADS, 1)
    shared_split_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ SharedParams p) {
  using C = sh::Cfg<D>;
  constexpr int NSTAGE = C::NSTAGE;
  constexpr int W_PROD = 8, W_MMA = 9;
  constexpr bool kBF16 = TileType<T>::kBF16;
  constexpr float NEG_INF = -INFINITY;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + C::SMEM_Q;
  uint64_t* full = reinterpret_cast<uint64_t*>(sKV + C::SMEM_KV);
  uint64_t* empty = full + NSTAGE;
  uint64_t* q_full = empty + NSTAGE;
  uint64_t* q_free = q_full + 1;   // a stretch's last S is there: Q may be overwritten
  uint64_t* s_full = q_free + 1;   // [2] of the warpgroups
  uint64_t* p_full = s_full + 2;   // [2]
  uint64_t* pv_done = p_full + 2;  // [2] a stretch's last P V of each warpgroup
  uint64_t* drain = pv_done + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile uint32_t* issued = reinterpret_cast<volatile uint32_t*>(abort_flag + 1);
  volatile uint32_t* tile_bad = issued + 1;  // [BAD_RING]
  static_assert(2 * C::NSTAGE * 8 + 9 * 8 + 12 + 4 * sh::BAD_RING <= C::SMEM_BAR, "barrier block");
  PlanScratch* scratch = reinterpret_cast<PlanScratch*>(sKV + C::SMEM_KV + C::SMEM_BAR);
  int* starts = reinterpret_cast<int*>(sKV + C::SMEM_KV + C::SMEM_BAR + C::SMEM_PLAN);
  static_assert(sizeof(PlanScratch) <= C::SMEM_PLAN, "plan scratch");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    mbar_init(q_full, 2 * sh::BM);
    mbar_init(q_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], sh::BM);
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

  SharedWalk w = shared_plan(p, starts, scratch);
  SharedSeg sg = {};
  // Rows of a stretch, and whether they make two row tiles.
  auto rows_of = [&](const SharedSeg& g) {
    return min(2 * sh::BM, w.s.rows - g.rt * 2 * sh::BM);
  };
  if (warp >= W_PROD) {
    regs_decrease<88>();
    if (warp == W_PROD) {
      // ============================ TMA producer ============================
      // Lane l < boxes * halves loads box l % boxes, half l / boxes of each tile.
      const int boxes = sh::BN / p.box;
      const int sub = lane % boxes, half = lane / boxes;
      const bool loads = half < C::HALVES;
      const uint64_t once = l2_policy_evict_first(), again = l2_policy_evict_last();
      uint32_t tc = 0;  // tiles so far: K at ring position 2 tc, V at 2 tc + 1
      bool ok = true;
      while (ok && shared_next(p, starts, w, &sg)) {
        const int32_t* table = p.page_table + (size_t)w.s.tab * p.max_pages;
        const int end = w.s.hi;
        const uint64_t pol = w.s.n_rt == 1 ? once : again;
        // Page of this lane's box in tile t (-1: nothing to load, -2: no such
        // page) and the row in it.
        auto page_of = [&](int t, int* pos) {
          const int row = t * sh::BN + sub * p.box;
          if (!loads || row >= end) return -1;
          const int pg = row / p.page_size;
          *pos = row - pg * p.page_size;
          const int id = table[pg];
          return id < 0 || id >= p.num_pages ? -2 : id;
        };
        auto load = [&](uint32_t cnt, const CUtensorMap* m, int id, int pos) {
          uint64_t* bar = &full[cnt % NSTAGE];
          const uint32_t bytes =
              __popc(__ballot_sync(0xffffffffu, id >= 0)) * (uint32_t)p.box * 128u;
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          if (id >= 0)
            tma_load_4d_hint(
                sKV + (cnt % NSTAGE) * C::TILE_BYTES + half * sh::HALF_BYTES + sub * p.box * 128,
                m, bar, half * 64, sg.hkv, pos, id, pol);
          if (lane == 0) *issued = cnt + 1;
        };
        auto slot_free = [&](uint32_t cnt) {
          return mbar_wait<true>(&empty[cnt % NSTAGE], ((cnt / NSTAGE) & 1) ^ 1, abort_flag,
                                 &g_shared_err, 1);
        };
        // Pages are looked up two tiles ahead.
        int pos = 0, pos_n = 0, pos_nn = 0;
        int id = page_of(sg.t, &pos), id_n = sg.n > 1 ? page_of(sg.t + 1, &pos_n) : -1;
        for (int j = 0; j < sg.n; ++j, ++tc) {
          const int id_nn = j + 2 < sg.n ? page_of(sg.t + j + 2, &pos_nn) : -1;
          if (!(ok = slot_free(2 * tc))) break;
          const uint32_t bad = __ballot_sync(0xffffffffu, id == -2 && half == 0);
          if (lane == 0) {
            if (bad) atomicOr(&g_shared_err, kErrBounds);
            tile_bad[tc % sh::BAD_RING] = bad;
          }
          load(2 * tc, &tmK, id, pos);
          if (!(ok = slot_free(2 * tc + 1))) break;
          load(2 * tc + 1, &tmV, id, pos);
          id = id_n;
          pos = pos_n;
          id_n = id_nn;
          pos_n = pos_nn;
        }
      }
      __syncwarp();
    } else if (warp == W_MMA) {
      // ============================ MMA issuer (lane 0) ============================
      if (lane == 0) {
        constexpr uint32_t IDESC_S = idesc_f16(sh::BM, sh::BN, kBF16, false);
        constexpr uint32_t IDESC_O = idesc_f16(sh::BM, D, kBF16, true);
        const uint64_t dq = sdesc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dk = sdesc_sw128(smem_u32(sKV), 16, 1024);
        const uint64_t dv = sdesc_sw128(smem_u32(sKV), sh::HALF_BYTES, 1024);
        const uint32_t sd_hi = (uint32_t)(dq >> 32);
        const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, v_lo = (uint32_t)dv;
        // S[buf] = Q[tile] K^T, over D / 16 steps.
        auto issue_s = [&](int tile, int buf, uint32_t cnt) {
          const uint32_t a0 = q_lo + tile * (C::TILE_BYTES >> 4);
          const uint32_t b0 = k_lo + (cnt % NSTAGE) * (C::TILE_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * sh::HALF_BYTES + (k & 3) * 32) >> 4;
            mma_ss_lh(tmem + C::COL_S + buf * 128, a0 + off, sd_hi, b0 + off, sd_hi, IDESC_S,
                      k > 0 ? 1u : 0u);
          }
          mma_commit(&s_full[buf]);
        };
        // O[i] (+)= P[i] V, over 128 / 16 steps.
        auto issue_pv = [&](int i, uint32_t cnt, bool add) {
          const uint32_t b0 = v_lo + (cnt % NSTAGE) * (C::TILE_BYTES >> 4);
#pragma unroll
          for (int k = 0; k < sh::BN / 16; ++k)
            mma_ts_lh(tmem + C::COL_O + i * D, tmem + C::COL_S + i * 128 + k * 8,
                      b0 + (uint32_t)((k * 16 * 128) >> 4), sd_hi, IDESC_O, add || k > 0 ? 1u : 0u);
        };
        uint32_t tc = 0, seg = 0, cw[2] = {0, 0};
        bool ok = true;
        auto landed = [&](uint32_t cnt, unsigned site) {
          ok = mbar_wait<false>(&full[cnt % NSTAGE], (cnt / NSTAGE) & 1, abort_flag, &g_shared_err,
                                site);
          tc_fence_after();
          return ok;
        };
        auto p_ready = [&](int i, uint32_t n) {
          ok = mbar_wait<false>(&p_full[i], n & 1, abort_flag, &g_shared_err, 6 + i);
          tc_fence_after();
          return ok;
        };
        while (ok && shared_next(p, starts, w, &sg)) {
          const int n = sg.n;
          if (!(ok = mbar_wait<false>(q_full, seg & 1, abort_flag, &g_shared_err, 2))) break;
          ++seg;
          tc_fence_after();
          if (!landed(2 * tc, 3)) break;
          if (rows_of(sg) > sh::BM) {  // two row tiles on every key tile
            issue_s(0, 0, 2 * tc);
            issue_s(1, 1, 2 * tc);
            mma_commit(&empty[(2 * tc) % NSTAGE]);
            if (n == 1) mma_commit(q_free);
            for (int j = 0; j < n; ++j, ++tc) {
              const uint32_t cv = 2 * tc + 1, ck = cv + 1;
              const bool more = j + 1 < n;
              if (!landed(cv, 4) || !p_ready(0, cw[0])) break;
              issue_pv(0, cv, j > 0);
              if (more) {
                if (!landed(ck, 5)) break;
                issue_s(0, 0, ck);
              } else {
                mma_commit(&pv_done[0]);
              }
              if (!p_ready(1, cw[1])) break;
              issue_pv(1, cv, j > 0);
              mma_commit(&empty[cv % NSTAGE]);
              if (more) {
                issue_s(1, 1, ck);
                mma_commit(&empty[ck % NSTAGE]);
                if (j + 2 == n) mma_commit(q_free);
              } else {
                mma_commit(&pv_done[1]);
              }
              ++cw[0];
              ++cw[1];
            }
          } else {  // one row tile: alternate key tiles
            issue_s(0, 0, 2 * tc);
            mma_commit(&empty[(2 * tc) % NSTAGE]);
            if (n > 1) {
              if (!landed(2 * tc + 2, 3)) break;
              issue_s(0, 1, 2 * tc + 2);
              mma_commit(&empty[(2 * tc + 2) % NSTAGE]);
            }
            if (n <= 2) mma_commit(q_free);
            for (int j = 0; j < n; ++j, ++tc) {
              const int i = j & 1;
              const uint32_t cv = 2 * tc + 1, ck = cv + 3;
              if (!landed(cv, 4) || !p_ready(i, i ? cw[1] : cw[0])) break;
              if (i)
                ++cw[1];
              else
                ++cw[0];
              issue_pv(i, cv, j > 1);
              mma_commit(&empty[cv % NSTAGE]);
              if (j + 2 < n) {
                if (!landed(ck, 5)) break;
                issue_s(0, i, ck);
                mma_commit(&empty[ck % NSTAGE]);
                if (j + 3 == n) mma_commit(q_free);
              } else {
                mma_commit(&pv_done[i]);
              }
            }
          }
        }
        // Every MMA issued here has completed before tensor memory is freed.
        mma_commit(drain);
        mbar_wait_drain(drain, 0);
      }
      __syncwarp();
    }
  } else {
    regs_increase<208>();
    // ======================= softmax and partials =======================
    const int i = warp >> 2, wq = warp & 3;
    const int tid = wq * 32 + lane;  // row within the tile, and V row it clears
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t tS = t_lane + C::COL_S + i * 128, tO = t_lane + C::COL_O + i * D;
    const float c = p.c;
    const float hide = c < 0.f ? -NEG_INF : NEG_INF;
    uint32_t tc = 0, cw = 0, done = 0, seg = 0;
    bool ok = true;
    // This thread's row of Q for a stretch (one row tile: the first warpgroup's).
    auto load_q = [&](const SharedSeg& g) {
      const int rows = rows_of(g), rr = i * sh::BM + tid;
      if (rows > sh::BM || i == 0) {
        int s;
        const bool real = rr < rows;
        const size_t qrow = real ? shared_qrow(p, w.s.row0, g.hkv, g.rt * 2 * sh::BM + rr, &s) : 0;
        put_q_row<D>(sQ + i * C::TILE_BYTES, tid, static_cast<const T*>(p.q) + qrow * D, real);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(q_full);
    };
    bool have = shared_next(p, starts, w, &sg);
    if (have) load_q(sg);
    while (have) {
      const int rows = rows_of(sg), n = sg.n;
      const bool dual = rows > sh::BM;
      const int kind = sg.kind;
      const int rr = dual ? i * sh::BM + tid : tid;
      const bool row_ok = rr < rows, warp_ok = rr - lane < rows;
      const int lo = w.s.lo, end = w.s.hi;
      // Keys [lo, lim) are this row's, [lo, end) somebody's; all rows see those below least.
      int lim = end, least = end;
      if (kind == 1) {
        int s = 0;
        if (row_ok) shared_qrow(p, 0, 0, sg.rt * 2 * sh::BM + rr, &s);
        least = end - p.Sq + 1;
        lim = least + s;
      }
      float m_used = NEG_INF, l = 0.f;
      for (int j = dual ? 0 : i; j < n; j += dual ? 1 : 2) {
        const uint32_t tj = tc + j;
        if (!(ok = mbar_wait<false>(&s_full[i], cw & 1, abort_flag, &g_shared_err, 8 + i))) break;
        ++cw;
        __syncwarp();
        tc_fence_after();
        const int kv0 = (sg.t + j) * sh::BN;
        const uint32_t bad = tile_bad[tj % sh::BAD_RING];
        const bool masked = kv0 < lo || kv0 > least - sh::BN || bad;
        if (masked) {
          // V rows that no query sees can hold anything: they are cleared, since 0 *
          // NaN in P V would reach every row.
          const Mask128 fine = sound_keys(bad, p.box);
          const uint32_t cv = 2 * tj + 1;
          if (!(ok = mbar_wait<false>(&full[cv % NSTAGE], (cv / NSTAGE) & 1, abort_flag,
                                      &g_shared_err, 10)))
            break;
          clear_rows<D>(sKV + (cv % NSTAGE) * C::TILE_BYTES, wq, lane,
                        Mask128{fine.lo & low_bits(end - kv0) & ~low_bits(lo - kv0),
                                fine.hi & low_bits(end - kv0 - 64) & ~low_bits(lo - kv0 - 64)});
        }
        if (warp_ok) {
          auto mask = [&](uint32_t (&sr)[4][32]) {
            const Mask128 fine = sound_keys(bad, p.box);
            hide_keys(sr,
                      Mask128{fine.lo & low_bits(lim - kv0) & ~low_bits(lo - kv0),
                              fine.hi & low_bits(lim - kv0 - 64) & ~low_bits(lo - kv0 - 64)},
                      hide);
          };
          // (S of this tile was issued after P V of this warpgroup's last: both are done.)
          auto settled = [] { return true; };
          softmax_tile<D, T>(tS, tO, c, j < (dual ? 1 : 2), masked, mask, settled, &m_used, &l);
        }
        tc_fence_before();
        mbar_arrive(&p_full[i]);
      }
      if (!ok) break;
      tc += n;
      const bool active = dual || i < n;
      const int half = dual ? sh::BM : p.half[kind];
      const size_t slot = (size_t)sg.id * 2 * p.half[kind] + i * half + tid;
      float4* const po = reinterpret_cast<float4*>(p.part_o[kind]) +
                         (size_t)sg.id * (D / 4) * 2 * p.half[kind] + i * half + tid;
      float2* const pml = reinterpret_cast<float2*>(p.part_ml[kind]) + slot;
      const size_t col = 2 * (size_t)p.half[kind];
      have = shared_next(p, starts, w, &sg);
      if (have) {
        if (!(ok = mbar_wait<false>(q_free, seg & 1, abort_flag, &g_shared_err, 11))) break;
        load_q(sg);
      }
      ++seg;
      if (!active) {
        if (row_ok) *pml = make_float2(NEG_INF, 0.f);
        continue;
      }
      if (!(ok = mbar_wait<false>(&pv_done[i], done & 1, abort_flag, &g_shared_err, 12))) break;
      ++done;
      __syncwarp();
      tc_fence_after();
      if (warp_ok) {
        if (row_ok) *pml = make_float2(m_used, l);
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(tO + q * 32, o);
          tmem_wait_ld();
          reg_fence32(o);
          if (!row_ok) continue;
          // [column / 4][row] of 16 bytes: the lanes' rows side by side.
#pragma unroll
          for (int x = 0; x < 8; ++x)
            po[(q * 8 + x) * col] =
                make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]),
                            __uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3]));
        }
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  // After an abort: every load that may still be in flight, before the CTA and its
  // shared memory go.
  if (warp == W_PROD && *abort_flag) {
    const uint32_t n = *issued;
    for (uint32_t u = n > (uint32_t)NSTAGE ? n - NSTAGE : 0u; u < n; ++u)
      mbar_wait_drain(&full[u % NSTAGE], (u / NSTAGE) & 1);
    __syncwarp();
  }
}

// Merge: a thread takes 16 columns of a row, the lanes of a warp 32 rows of one kv
// head, so that loads are as wide as the split kernel's stores.  A row has the
// partials of its group's unit and of its own, walked strip by strip, the next
// partial's loads ahead of this one's sums.  KS = 1: a thread walks all of them.
// KS = 8: the block's 8 warps share one set of 32 rows x 16 columns, each every 8th
// strip.
constexpr int kJoinWarps = 8;
template <int D, typename T, int KS>
__global__ void __launch_bounds__(kJoinWarps * 32)
    shared_merge_kernel(const __grid_constant__ SharedParams p) {
  pdl_launch_dependents();
  pdl_wait_primary();
  constexpr int NC = D / 16;  // column chunks of a row
  __shared__ float sM[KS > 1 ? KS : 1][32], sDen[KS > 1 ? KS : 1][32];
  __shared__ float sAcc[KS > 1 ? KS : 1][16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int all_rows = p.B * p.SqG, sets = (all_rows + 31) / 32;
  int x, chunk;
  if constexpr (KS == 1) {
    x = blockIdx.x * (kJoinWarps / NC) + warp / NC;
    chunk = warp % NC;
    if (x >= sets * p.Hkv) return;
  } else {
    x = blockIdx.x / NC;
    chunk = blockIdx.x - x * NC;
  }
  const int hkv = x / sets, R = (x - hkv * sets) * 32 + lane;
  const bool real = R < all_rows;
  const int owners = p.groups + p.B;
  const long long total = p.first[owners];
  const int W = (int)p.first[owners + 1], slack = (int)p.first[owners + 2],
            groups = (int)p.first[owners + 3];
  const long long ctas = total < p.ctas ? total : p.ctas;
  float M = -INFINITY, den = 0.f, acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  // The partial whose loads are under way.
  float2 ml = make_float2(-INFINITY, 0.f);
  float4 ov[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) ov[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto join = [&](float2 a, const float4 (&v)[4]) {
    if (!(a.y > 0.f || a.y != a.y)) return;  // saw no key  (NaN joins)
    float wt;
    if (a.x > M) {
      const float f = M == -INFINITY ? 0.f : fast_exp2(M - a.x);
      den *= f;
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] *= f;
      M = a.x;
      wt = 1.f;
    } else {
      wt = fast_exp2(a.x - M);
    }
    den += wt * a.y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[4 * e] += wt * v[e].x;
      acc[4 * e + 1] += wt * v[e].y;
      acc[4 * e + 2] += wt * v[e].z;
      acc[4 * e + 3] += wt * v[e].w;
    }
  };
  auto take = [&](int kind, long long id, int at) {
    const size_t half2 = 2 * (size_t)p.half[kind];
    const float2 a = reinterpret_cast<const float2*>(p.part_ml[kind])[id * half2 + at];
    const float4* src = reinterpret_cast<const float4*>(p.part_o[kind]) +
                        ((size_t)id * (D / 4) + chunk * 4) * half2 + at;
    float4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = src[e * half2];
    join(ml, ov);
    ml = a;
#pragma unroll
    for (int e = 0; e < 4; ++e) ov[e] = v[e];
  };
  // The CTA whose range holds place y: the largest c with total * c / ctas <= y.
  auto cta_of = [&](long long y) {
    return (int)quotient((y + 1) * ctas - 1, total);
  };
  auto walk = [&](int o, int kind, int r) {  // all partials of row r of owner o
    const Shape s = shape_of(p, p.starts, groups, o, W);
    if (s.T == 0) return;
    const int rt = r / (2 * sh::BM), rr = r - rt * 2 * sh::BM;
    const bool dual = min(2 * sh::BM, s.rows - rt * 2 * sh::BM) > sh::BM;
    const long long head = p.first[o] + hkv * places_per_head(s, slack);
    for (int k = KS > 1 ? warp : 0; k < s.S; k += KS) {
      const int len = min(s.len, s.T - k * s.len);
      const long long y = head + (long long)k * s.n_rt * (s.len + slack) + (long long)rt * (len + slack);
      const int c0 = cta_of(y), c1 = cta_of(y + len - 1);
      const long long id = (long long)p.pieces[o] + (hkv * s.S + k) * s.n_rt + rt;
      for (int c = c0; c <= c1; ++c) {
        take(kind, id + c, rr);
        if (!dual) take(kind, id + c, rr + p.half[kind]);
      }
    }
  };
  size_t row = 0;
  if (real) {
    const int b = R / p.SqG, r = R - b * p.SqG, s = r / p.G;
    row = ((size_t)b * p.Sq + s) * p.Hq + (size_t)hkv * p.G + (r - s * p.G);
    const int L = shared_len(p, b);
    if (covered(p, p.starts, groups, b, L) > 0) {
      const int g = group_of(p.starts, groups, b);
      walk(g, 0, (b - p.starts[g]) * p.SqG + r);
    }
    walk(p.groups + b, 1, r);
    join(ml, ov);
  }
  T* const dst = static_cast<T*>(p.o) + row * D + chunk * 16;
  if constexpr (KS > 1) {
    // The warps' results meet in shared memory; then each warp finishes two of the
    // 16 columns.
    sM[warp][lane] = M;
    sDen[warp][lane] = den;
#pragma unroll
    for (int e = 0; e < 16; ++e) sAcc[warp][e][lane] = acc[e];
    __syncthreads();
    static_assert(KS == 1 || (KS == kJoinWarps && 2 * KS == 16), "two columns per warp");
    M = -INFINITY;
#pragma unroll
    for (int i = 0; i < KS; ++i) M = fmaxf(M, sM[i][lane]);
    float a0 = 0.f, a1 = 0.f;
    den = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const float m = sM[i][lane];
      const float wt = m == -INFINITY && !(sDen[i][lane] != sDen[i][lane]) ? 0.f : fast_exp2(m - M);
      den += wt * sDen[i][lane];
      a0 += wt * sAcc[i][2 * warp][lane];
      a1 += wt * sAcc[i][2 * warp + 1][lane];
    }
    if (!real) return;
    const float inv = den == 0.f ? 0.f : 1.f / den;
    reinterpret_cast<uint32_t*>(dst)[warp] = TileType<T>::pack(a0 * inv, a1 * inv);
    if (warp != 0) return;
  } else {
    if (!real) return;
    const float inv = den == 0.f ? 0.f : 1.f / den;
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

// A cache without capacity: no row sees a key.
__global__ void shared_zero_kernel(uint16_t* o, size_t n, float* lse, size_t nl) {
  const size_t at = blockIdx.x * (size_t)blockDim.x + threadIdx.x;
  const size_t step = (size_t)gridDim.x * blockDim.x;
  for (size_t i = at; i < n; i += step) o[i] = 0;
  if (lse)
    for (size_t i = at; i < nl; i += step) lse[i] = -INFINITY;
}

template <int D, typename T>
static cudaError_t launch_shared(const SharedParams& p, const CUtensorMap& tk,
                                 const CUtensorMap& tv, cudaStream_t stream) {
  using C = sh::Cfg<D>;
  static int attr_set[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE)) {
    e = cudaFuncSetAttribute(shared_split_kernel<D, T>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_TOTAL);
    if (e != cudaSuccess) return e;
    // As in the tree decode: the merge keeps the split kernel's division of the SM.
    for (auto k : {shared_merge_kernel<D, T, 1>, shared_merge_kernel<D, T, kJoinWarps>}) {
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
  cfg.gridDim = dim3((unsigned)p.ctas, 1, 1);
  cfg.blockDim = dim3(sh::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_TOTAL;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, shared_split_kernel<D, T>, tk, tv, p);
  if (e != cudaSuccess) return e;
  constexpr int NC = D / 16;
  const long long sets = ((long long)p.B * p.SqG + 31) / 32 * p.Hkv;
  const bool split = sets * NC <= 4 * p.ctas;
  return split ? launch_dependent(shared_merge_kernel<D, T, kJoinWarps>, dim3((unsigned)(sets * NC)),
                                  kJoinWarps * 32, stream, p)
               : launch_dependent(shared_merge_kernel<D, T, 1>,
                                  dim3((unsigned)((sets * NC + kJoinWarps - 1) / kJoinWarps)),
                                  kJoinWarps * 32, stream, p);
}

int set_shared_wait_limit(unsigned long long ns) { return set_wait_limit_this_unit(ns); }

int read_shared_error(unsigned int* out, int reset) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_shared_err, sizeof(v));
  if (e != cudaSuccess) return e;
  if (reset && v) {
    const unsigned int z = 0;
    e = cudaMemcpyToSymbol(g_shared_err, &z, sizeof(z));
    if (e != cudaSuccess) return e;
  }
  *out = v;
  return cudaSuccess;
}

}  // namespace fa

static bool al(const void* p, unsigned n) {
  return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

extern "C" int fa_decode_shared_fwd(const void* q, const void* kpages, const void* vpages,
                                    const int32_t* page_table, const int32_t* seqlens,
                                    const int32_t* group_starts, const int32_t* prefix_lens,
                                    void* o, float* lse, int B, int Sq, int Hq, int Hkv,
                                    int num_pages, int page_size, int max_pages, int groups,
                                    int D, float scale, int dtype, cudaStream_t stream) {
  if (B < 0 || Sq < 0 || Hq < 0 || Hkv < 0 || num_pages < 0 || max_pages < 0 || groups < 0)
    return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_INVALID_ARG;
  if (!isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (page_size < 32 || page_size % 32 != 0) return FA_ERR_INVALID_ARG;
  if (groups > fa::sh::MAX_GROUPS) return FA_ERR_UNSUPPORTED;
  if (B == 0 || Sq == 0 || Hq == 0) return FA_OK;
  if (Hkv == 0 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  // Row indexes and the merge's grid (at most one block per row) fit 31 bits.
  if ((int64_t)B * Sq * Hq > INT32_MAX) return FA_ERR_INVALID_ARG;
  if ((int64_t)max_pages * page_size > INT32_MAX) return FA_ERR_INVALID_ARG;
  if (!al(q, 16) || !al(o, 16)) return FA_ERR_INVALID_ARG;
  if (lse && !al(lse, 4)) return FA_ERR_INVALID_ARG;
  if (!al(seqlens, 4)) return FA_ERR_INVALID_ARG;
  if (groups > 0 && (!al(group_starts, 4) || !al(prefix_lens, 4))) return FA_ERR_INVALID_ARG;
  if (max_pages > 0 &&
      (num_pages < 1 || !al(kpages, 16) || !al(vpages, 16) || !al(page_table, 4)))
    return FA_ERR_INVALID_ARG;
  if ((int64_t)num_pages * page_size > (1ll << 40) / (2 * D) / Hkv) return FA_ERR_INVALID_ARG;
  const fa::SetupDuringCapture setup;
  if (max_pages == 0) {
    const size_t rows = (size_t)B * Sq * Hq, n = rows * D;
    fa::shared_zero_kernel<<<(unsigned)((n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096), 256, 0,
                             stream>>>(static_cast<uint16_t*>(o), n, lse, rows);
    return fa::record_cuda_status(cudaGetLastError(), "shared decode zero-fill launch");
  }
  fa::SharedParams p = {};
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.page_table = page_table;
  p.seqlens = seqlens;
  p.starts = group_starts;
  p.prefix = prefix_lens;
  p.B = B;
  p.groups = groups;
  p.Sq = Sq;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.SqG = Sq * p.G;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  // Keys per TMA box: a tile's boxes must not straddle pages.
  p.box = page_size % 128 == 0 ? 128 : (page_size % 64 == 0 ? 64 : 32);
  p.c = scale * 1.4426950408889634f;
  // scale == 0: every visible score is 0; a tiny c keeps hidden keys at -inf.
  if (p.c == 0.f) p.c = 1e-30f;
  p.ctas = fa::sm_count() > 0 ? fa::sm_count() : 148;
  // Slots: every piece, and one more for each boundary between CTAs' ranges.  Pieces:
  // one per (row-tile pair, kv head), and strips, of which all have at most one per CTA
  // beyond those.
  const long long rows_all = (long long)B * p.SqG, pair = 2 * fa::sh::BM;
  const long long units[2] = {
      groups > 0 ? (groups < B / 2 ? groups : B / 2) + rows_all / pair : 0,
      (long long)B * ((p.SqG + pair - 1) / pair)};
  size_t slots[2], bytes = 0, at_o[2], at_ml[2];
  const size_t owners = (size_t)groups + B;
  bytes = (owners + 4) * sizeof(long long) + (owners * sizeof(int) + 31) / 32 * 32;
  bytes = (bytes + 255) / 256 * 256;
  for (int k = 0; k < 2; ++k) {
    const long long rows = k == 0 ? rows_all : p.SqG;
    p.half[k] = (int)(rows < fa::sh::BM ? rows : fa::sh::BM);
    slots[k] = k == 0 && groups == 0 ? 0 : (size_t)units[k] * Hkv + 2 * (size_t)p.ctas;
    at_o[k] = bytes;
    bytes += slots[k] * D * 2 * p.half[k] * sizeof(float);
    at_ml[k] = bytes;
    bytes += slots[k] * 2 * 2 * p.half[k] * sizeof(float);
    bytes = (bytes + 255) / 256 * 256;
  }
  CUtensorMap tk, tv;
  if (fa::encode_tmap_rows(&tk, kpages, D, Hkv, page_size, num_pages, p.box) ||
      fa::encode_tmap_rows(&tv, vpages, D, Hkv, page_size, num_pages, p.box))
    return fa::record_cuda_status(cudaErrorInvalidValue, "shared decode tensor maps");
  void* scratch = nullptr;
  cudaError_t e = fa::scratch_alloc(&scratch, bytes, stream);
  if (e != cudaSuccess) return fa::record_cuda_status(e, "shared decode scratch");
  uint8_t* const base = static_cast<uint8_t*>(scratch);
  p.first = reinterpret_cast<long long*>(base);
  p.pieces = reinterpret_cast<int*>(base + (owners + 4) * sizeof(long long));
  for (int k = 0; k < 2; ++k) {
    p.part_o[k] = reinterpret_cast<float*>(base + at_o[k]);
    p.part_ml[k] = reinterpret_cast<float*>(base + at_ml[k]);
  }
  const bool bf16 = dtype == FA_BF16;
  if (D == 64)
    e = bf16 ? fa::launch_shared<64, __nv_bfloat16>(p, tk, tv, stream)
             : fa::launch_shared<64, __half>(p, tk, tv, stream);
  else
    e = bf16 ? fa::launch_shared<128, __nv_bfloat16>(p, tk, tv, stream)
             : fa::launch_shared<128, __half>(p, tk, tv, stream);
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  if (e != cudaSuccess) return fa::record_cuda_status(e, "shared decode launch");
  return fa::record_cuda_status(ef, "shared decode cudaFreeAsync");
}
