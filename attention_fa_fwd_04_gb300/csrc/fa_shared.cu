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
// against a range of keys.
//   Units of many rows (groups; sequences of more than 16 rows) are done by tcgen05
//   MMAs against 128-key tiles as in the tree decode (S and O in tensor memory, P
//   written back over S).  A CTA has two softmax warpgroups, one TMA producer warp and
//   one MMA warp.  Units of more than 128 rows give each warpgroup a 128-row tile, and
//   both meet every key tile; with fewer rows the warpgroups take alternate key tiles of
//   the one row tile, each with sums of its own, so that the softmax of one runs beside
//   the other's.
//   Sequences of up to 16 rows are a stream of their own keys: each of six warps of a
//   CTA streams a range of its own through two tiles of 32 keys in shared memory and
//   multiplies by mma.sync (keys as M, rows as N).  No warp waits for another, so the
//   ends of short ranges cost nothing but themselves.
// Split: lengths, prefixes and groups are device data.  The units of either kind form a
// list of tiles; the CTAs are shared out between the lists by what they cost, and a list
// is cut into equal ranges, one per CTA (one per warp).  A unit of several row-tile
// pairs whose keys are more than L2 keeps is cut into strips about as long as a range,
// and the pairs of one strip stand side by side in the list, so that the CTAs which read
// the same keys do so at the same time and share them through L2.  Every stretch of a
// range leaves a partial; a second kernel merges a row's.  Every CTA makes the lists for
// itself, from the lengths; in the first kind of CTA one warp walks its range and tells
// the others stretch by stretch, ahead of them.
//
// Measured (both kernels, device time in a captured sequence; floor): 64 sequences of 8 rows
// per kv head behind 8192 tokens 52 to 64 us over several boxes and inputs (31.5), 32 of 16 rows
// behind 65536 145 to 148 (73.4: 956 TFLOP/s and 3.0 TB/s together; 169 where calls follow each
// other with nothing between, whose CTAs start under the merge of the call before), 48 of 16
// rows in 5 groups, D = 64, 30.1 (4.2), 8 of 4 rows behind 1500 17.6 (0.4), 128 of 32 rows behind
// 128 with up to 100 keys of their own 78 (7.3).  At D = 128 the split kernel spills 96 bytes of
// stores in 168 registers.  What bounds it: with many rows the softmax (two 128-row tiles per
// key tile take 1.76 us, their MMAs 1.34) on the SMs of the prefixes and the stream on the
// others; with few, the lists (4 us), the first tiles (8) and the merge (4 to 10).
#include <math.h>

#include <type_traits>

#include "fa.h"
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_shares.h"
#include "fa_tiles.cuh"

namespace fa {

__device__ unsigned int g_shared_err = 0;

namespace sh {
using namespace tiles;
constexpr int MAX_GROUPS = 1024;  // their starts and prefixes lie in shared memory
constexpr int THREADS = 384;
constexpr int WARPS = THREADS / 32;
constexpr int KEPT = THREADS;  // owners whose keys a CTA keeps in shared memory
// Places that a 128-key tile takes in its list, so that equal ranges take equal times: one
// that two row tiles meet (1.45 us), or one row tile in turns; and places without a tile
// after each piece, for what a stretch costs beside its tiles.  A 32-key tile of a few
// rows is one place of the other list.
constexpr int COST = 3, SLACK = 4, SLACK_FEW = 2;
constexpr int FEW = 16;       // rows that a warp streams keys for
constexpr int FEW_WARPS = 6;  // such warps of a CTA
constexpr int FEW_KEYS = 32;  // keys of their tiles
constexpr int RING = 4;        // stretches told ahead
constexpr long long L2_KEEPS = 48 << 20;  // bytes of a unit's K/V, over all kv heads

// A stretch of one unit's tiles.
struct Seg {
  int kind;      // 0 group, 1 sequence, -1 the end
  int hkv;
  int r0, rows;  // first query row within the unit, rows: up to 256
  int t, n;      // first tile, tiles
  int id;        // partial
  int lo, hi;    // keys [lo, hi)
  int row0;      // first sequence
  int tab;       // sequence whose row of the page table lists the keys
  int twice;     // other rows meet the same keys: worth keeping in L2
};

// A unit's tiles.
struct Shape {
  int t0, T;   // first tile and tiles
  int n_rt;    // pairs of row tiles
  int cost;    // places of a tile
  int S, len;  // strips, tiles of each but the last
};

// What every CTA finds out about the list, in shared memory.
struct Plan {
  long long sums[2 * WARPS];
  long long x, hi;  // this CTA's range of places
  long long first;  // first place of owner o
  int o, piece0;    // owner; pieces of its kind before it
  Shape s;          // and its tiles
  int W, slack, groups;
  int range, few;   // this CTA's (first) range; whether its warps stream
  int used;         // ranges of the streaming warps
  long long total[2];
  int lo[KEPT], end[KEPT], tab[KEPT], len[KEPT];
  int starts[MAX_GROUPS + 1], prefix[MAX_GROUPS];
};

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE_BYTES = HALVES * HALF_BYTES;
  static constexpr int NSTAGE = D == 128 ? 4 : 10;  // K and V tiles in flight
  static constexpr int SMEM_Q = 2 * TILE_BYTES;
  static constexpr int SMEM_KV = NSTAGE * TILE_BYTES;
  static constexpr int SMEM_BAR = 512, SMEM_RING = FEW_WARPS * 288;  // (told stretches)
  static_assert(RING * 64 <= SMEM_RING, "a ring, or a walk per streaming warp");
  static_assert(sizeof(Seg) <= 64 && alignof(Seg) <= 64, "a stretch's slot");
  static constexpr int SMEM_TOTAL = 1024 + SMEM_Q + SMEM_KV +
                                    SMEM_BAR + SMEM_RING + (int)sizeof(Plan);
  static_assert(SMEM_TOTAL <= 227 * 1024, "shared memory per CTA");
  static_assert(NSTAGE / 2 + 2 < BAD_RING, "tiles in flight");
  // Streaming warps: two tiles each, K and V.
  static constexpr int FEW_HALF = FEW_KEYS * 128, FEW_KV = HALVES * FEW_HALF;
  static_assert(FEW_WARPS * 4 * FEW_KV <= SMEM_Q + SMEM_KV, "streaming warps' tiles");
  // Tensor memory: S of each warpgroup, then O of each.
  static constexpr uint32_t COL_S = 0, COL_O = 256, TMEM_COLS = 512;
};
}  // namespace sh

// Owners of units: group g is owner g, sequence b owner groups + b.  What the merge
// knows of them.
struct __align__(16) SharedOwner {
  long long first;  // first place
  int piece0;       // pieces of its kind before it
  int lo, hi;       // keys [lo, hi)
  int row0, rows;   // first sequence, query rows per kv head
  int group;        // of a sequence that its group's unit covers, else -1
};
// ... and of the list.
struct SharedList {
  long long total[2];   // places of the two kinds' lists
  int used[2];          // ranges of each
  int W, slack[2];
};

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
  int half[2];  // rows of a warpgroup in a slot
  int share_few;  // what a place of the streamed list costs, to SHARE_MANY
  int few;      // sequences are streamed by warps; their partials: [id][SqG][D], [id][SqG][2]
  SharedOwner* owner;  // [groups + B]
  SharedList* list;
  int B, groups, Sq, Hq, Hkv, G, SqG;
  int page_size, max_pages, num_pages, box, ctas;
  long long keep_tiles;  // tiles of a unit, all kv heads, that L2 keeps
  float c;  // scale * log2(e)
  int merge_rows;  // of a merge block
};

// Several pairs of row tiles against more keys than L2 keeps.
__device__ __forceinline__ bool can_be_cut(const SharedParams& p, const sh::Shape& s) {
  return s.n_rt > 1 && (long long)s.T * p.Hkv > p.keep_tiles;
}
__device__ __forceinline__ sh::Shape shape_of(const SharedParams& p, bool few, int rows, int lo, int hi,
                                          int W) {
  sh::Shape s;
  const int keys = few ? sh::FEW_KEYS : sh::BN;
  s.t0 = lo / keys;
  s.T = hi > lo ? (int)(((uint32_t)hi + keys - 1) / keys) - s.t0 : 0;
  s.n_rt = (rows + 2 * sh::BM - 1) / (2 * sh::BM);
  s.cost = few ? 1 : sh::COST;
  s.S = 1;
  s.len = s.T;
  if (can_be_cut(p, s) && s.T > W) {
    const uint32_t S = ((uint32_t)s.T + W / 2) / (uint32_t)W;
    s.len = (int)(((uint32_t)s.T + S - 1) / S);
    s.S = (s.T + s.len - 1) / s.len;
  }
  return s;
}
__device__ __forceinline__ long long places_per_head(const sh::Shape& s, int slack) {
  return s.T > 0 ? (long long)s.n_rt * ((long long)s.T * s.cost + (long long)s.S * slack) : 0;
}
__device__ __forceinline__ long long pieces_of(const SharedParams& p, const sh::Shape& s) {
  return s.T > 0 ? (long long)p.Hkv * s.S * s.n_rt : 0;
}

__device__ __forceinline__ long long shared_cap(const SharedParams& p) {
  return (long long)p.max_pages * p.page_size;
}
__device__ __forceinline__ int shared_len(const SharedParams& p, int b) {
  const int L = p.seqlens[b];
  return L < 0 ? 0 : (L > shared_cap(p) ? (int)shared_cap(p) : L);
}
__device__ __forceinline__ int kept_len(const SharedParams& p, const sh::Plan* pl, int b) {
  return b < sh::KEPT ? pl->len[b] : shared_len(p, b);
}
// Tokens that group g shares: 0 for fewer than two members.
__device__ __forceinline__ int group_prefix(const SharedParams& p, const sh::Plan* pl, int g) {
  if (pl->starts[g + 1] - pl->starts[g] < 2) return 0;
  const int P = pl->prefix[g];
  return P < 0 || P > shared_cap(p) ? 0 : P;
}
// The group of sequence b, or -1.
__device__ __forceinline__ int group_of(const sh::Plan* pl, int b) {
  if (pl->groups == 0 || b < pl->starts[0] || b >= pl->starts[pl->groups]) return -1;
  int lo = 0, hi = pl->groups;  // starts[lo] <= b < starts[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pl->starts[mid] <= b)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}
// An owner's rows and keys: a group's prefix, read through the first member that is
// past it (none: no keys); of a sequence what its group's unit does not cover: the
// keys behind the prefix, or all of one that is not past it.
struct Keys {
  int lo, hi, tab, row0, rows, group;
};
__device__ __forceinline__ Keys keys_of(const SharedParams& p, const sh::Plan* pl, int o) {
  Keys k;
  if (o < p.groups) {
    const bool real = o < pl->groups;
    k.lo = 0;
    k.hi = real ? group_prefix(p, pl, o) : 0;
    k.row0 = real ? pl->starts[o] : 0;
    k.rows = real ? (pl->starts[o + 1] - pl->starts[o]) * p.SqG : 0;
    k.tab = k.row0;
    k.group = -1;
    if (k.hi > 0) {
      while (k.tab < pl->starts[o + 1] && kept_len(p, pl, k.tab) - p.Sq + 1 < k.hi) ++k.tab;
      if (k.tab == pl->starts[o + 1]) k.hi = 0;
    }
  } else {
    const int b = o - p.groups;
    k.row0 = k.tab = b;
    k.rows = p.SqG;
    k.hi = kept_len(p, pl, b);
    k.lo = 0;
    k.group = group_of(pl, b);
    if (k.group >= 0) {
      const int P = group_prefix(p, pl, k.group);
      if (k.hi - p.Sq + 1 >= P) k.lo = P;
    }
    if (k.lo == 0) k.group = -1;
  }
  return k;
}

// Inclusive sums of a and b over the block, and the totals.
__device__ __forceinline__ void block_sums(long long& a, long long& b, long long* sums,
                                           long long* ta, long long* tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
    sums[2 * warp] = a;
    sums[2 * warp + 1] = b;
  }
  __syncthreads();
  // Every warp adds the warps' totals up for itself.
  long long x = lane < sh::WARPS ? sums[2 * lane] : 0, y = lane < sh::WARPS ? sums[2 * lane + 1] : 0;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  *ta = __shfl_sync(0xffffffffu, x, sh::WARPS - 1);
  *tb = __shfl_sync(0xffffffffu, y, sh::WARPS - 1);
  const long long pa = __shfl_sync(0xffffffffu, x, warp ? warp - 1 : 0),
                  pb = __shfl_sync(0xffffffffu, y, warp ? warp - 1 : 0);
  if (warp) {
    a += pa;
    b += pb;
  }
}

// Block-wide: the list, and this CTA's range of it, into *pl.  CTA 0 also writes it
// down for the merge.
__device__ __forceinline__ void shared_plan(const SharedParams& p, sh::Plan* pl) {
  const int t = threadIdx.x;
  const int owners = p.groups + p.B;
  if (t == 0) {
    pl->o = -1;
    pl->groups = p.groups;
  }
  // Starts, prefixes and lengths at once.
  for (int b = t; b < p.B && b < sh::KEPT; b += sh::THREADS) pl->len[b] = shared_len(p, b);
  bool odd = false, far = false;
  for (int i = t; p.groups > 0 && i <= p.groups; i += sh::THREADS) {
    const int s = p.starts[i];
    odd |= s < 0 || s > p.B || (i > 0 && s < p.starts[i - 1]);
    pl->starts[i] = s;
    if (i < p.groups) {
      const int P = p.prefix[i];
      far |= P < 0 || P > shared_cap(p);
      pl->prefix[i] = P;
    }
  }
  odd = __syncthreads_or(odd);
  if (odd) {
    if (t == 0) pl->groups = 0;
    __syncthreads();
  }
  if (blockIdx.x == 0 && (far || (odd && t == 0))) atomicOr(&g_shared_err, kErrBounds);
  // Places of the tiles in the lists: of the groups, and of the sequences where warps
  // stream them, else all in the first.
  auto few = [&](int o) { return p.few && o >= p.groups; };
  auto pieces_at = [&](int o, const sh::Shape& s) {
    return o < p.groups ? pieces_of(p, s) << 32 : pieces_of(p, s);
  };
  // With an owner per thread, sums of tiles and pieces (groups' in the upper half) up to
  // each owner; else the tiles of either kind.
  const bool one = owners <= sh::THREADS;
  Keys mine = {};  // of this thread's first owner
  long long tiles[2] = {0, 0}, all_tiles[2], my_tiles = 0, my_pieces = 0, all_pieces = 0;
  sh::Shape whole = {};
  bool cut = false;  // into strips
  for (int o = t; o < owners; o += sh::THREADS) {
    const Keys k = keys_of(p, pl, o);
    if (o == t) {
      mine = k;
      pl->lo[o] = k.lo;
      pl->end[o] = k.hi;
      pl->tab[o] = k.tab;
    }
    const sh::Shape s = shape_of(p, few(o), k.rows, k.lo, k.hi, INT32_MAX);
    tiles[few(o)] += (long long)p.Hkv * s.n_rt * s.T * s.cost;
    if (one) {
      my_pieces = pieces_at(o, s);
      whole = s;
    }
    cut |= can_be_cut(p, s);
  }
  long long sum_tiles = my_tiles = tiles[0] + tiles[1], sum_pieces = my_pieces;
  if (one) {
    if (t == 0) pl->total[0] = 0;
    block_sums(sum_tiles, sum_pieces, pl->sums, &all_tiles[1], &all_pieces);
    if (t == p.groups - 1) pl->total[0] = sum_tiles;
    cut = __syncthreads_or(cut);
    all_tiles[0] = p.few ? pl->total[0] : all_tiles[1];
    all_tiles[1] -= all_tiles[0];
  } else {
    block_sums(tiles[0], tiles[1], pl->sums, &all_tiles[0], &all_tiles[1]);
  }
  const int n = p.ctas;
  // CTAs of the first kind, for lists of a and z places.
  auto share = [&](long long a, long long z, long long starts) {
    return sh::ctas_of_tiles(a, z, starts, n, p.share_few);
  };
  const long long per = (long long)max(1, share(all_tiles[0], all_tiles[1], 0)) * sh::COST;
  const long long width = quotient(all_tiles[0] + per - 1, per);
  const int W = width < 1 ? 1 : (width > INT32_MAX ? INT32_MAX : (int)width);
  const int slack[2] = {all_tiles[0] > (long long)n * sh::COST ? sh::SLACK : 0,
                        all_tiles[1] > (long long)n * sh::FEW_WARPS ? sh::SLACK_FEW : 0};
  auto places_at = [&](int o, const Keys& k) {
    return p.Hkv * places_per_head(shape_of(p, few(o), k.rows, k.lo, k.hi, W), slack[few(o)]);
  };
  // Sums of places up to each owner; with an owner per thread they are those of the list
  // (a piece each where nothing is cut), else they are made again chunk by chunk.
  long long total[2], my_places = 0, sum_places = 0;
  if (one && !cut) {
    const long long of_groups = all_pieces >> 32, of_seqs = all_pieces & 0xffffffffll;
    const long long g = sum_pieces >> 32, q = sum_pieces & 0xffffffffll;
    total[0] = all_tiles[0] + slack[0] * (of_groups + (p.few ? 0 : of_seqs));
    total[1] = p.few ? all_tiles[1] + slack[1] * of_seqs : 0;
    my_places = my_tiles + slack[few(t)] * (t < p.groups ? my_pieces >> 32 : my_pieces);
    sum_places = few(t) ? total[0] + (sum_tiles - all_tiles[0]) + slack[1] * q
                        : sum_tiles + slack[0] * (g + q);
  } else if (one) {
    if (t < owners) {
      my_places = places_at(t, mine);
      my_pieces = pieces_at(t, shape_of(p, few(t), mine.rows, mine.lo, mine.hi, W));
    }
    sum_places = my_places;
    sum_pieces = my_pieces;
    __syncthreads();
    if (t == 0) pl->total[0] = 0;
    block_sums(sum_places, sum_pieces, pl->sums, &total[1], &all_pieces);
    if (t == p.groups - 1) pl->total[0] = sum_places;
    __syncthreads();
    total[0] = p.few ? pl->total[0] : total[1];
    total[1] -= total[0];
  } else {
    long long a = 0, z = 0;
    for (int o = t; o < owners; o += sh::THREADS) {
      const long long x = places_at(o, o == t ? mine : keys_of(p, pl, o));
      if (few(o))
        z += x;
      else
        a += x;
    }
    block_sums(a, z, pl->sums, &total[0], &total[1]);
  }
  // CTAs of either kind by what their lists cost.  Ranges in use are each as long as a tile
  // at least, so that every one of them between the first and the last of a piece holds a
  // tile of it.
  // (Units of a tile or two cost their starts too where they have no places for them: 64
  // sequences with a token each behind 8192 43 us, 56 without; 32 with 30 tokens behind 65536
  // 128 and 260.)
  const int many = share(total[0], total[1],
                         one && slack[1] == 0 ? sh::SLACK_FEW * (all_pieces & 0xffffffffll) : 0);
  const long long most = quotient(total[0], 2 * sh::COST);
  const int used[2] = {most < 1 ? 1 : (int)min(most, (long long)max(many, 1)),
                       (int)max(1ll, min(total[1], (long long)(n - many) * sh::FEW_WARPS))};
  const int kind = (int)blockIdx.x >= many;
  const int range = kind ? ((int)blockIdx.x - many) * sh::FEW_WARPS : (int)blockIdx.x;
  const long long base = kind ? total[0] : 0;
  const bool in_use = range < used[kind] && total[kind] > 0;
  const long long x = in_use ? base + quotient(total[kind] * range, used[kind]) : 0;
  const long long hi = in_use ? base + quotient(total[kind] * (range + 1), used[kind]) : 0;
  long long places0 = 0, pieces0 = 0;
  for (int o0 = 0; o0 < owners; o0 += sh::THREADS) {
    const int o = o0 + t;
    Keys k = mine;
    long long end_places = 0, end_pieces = 0;
    if (!one) {
      if (o0 > 0 && o < owners) k = keys_of(p, pl, o);
      my_places = my_pieces = 0;
      if (o < owners) {
        my_places = places_at(o, k);
        my_pieces = pieces_at(o, shape_of(p, few(o), k.rows, k.lo, k.hi, W));
      }
      sum_places = my_places;
      sum_pieces = my_pieces;
      block_sums(sum_places, sum_pieces, pl->sums, &end_places, &end_pieces);
    }
    const long long first = places0 + sum_places - my_places, before = pieces0 + sum_pieces - my_pieces;
    const int piece0 = (int)(o < p.groups ? before >> 32 : before & 0xffffffffll);
    if (o < owners) {
      if (first <= x && x < first + my_places && x < hi) {
        pl->o = o;
        pl->first = first;
        pl->piece0 = piece0;
        pl->s = one && !cut ? whole : shape_of(p, few(o), k.rows, k.lo, k.hi, W);
      }
      if (blockIdx.x == 0)
        p.owner[o] = SharedOwner{first - (few(o) ? total[0] : 0), piece0, k.lo, k.hi, k.row0, k.rows,
                                 k.group};
    }
    places0 += end_places;
    pieces0 += end_pieces;
    if (blockIdx.x != 0 && places0 > x) break;  // (block-uniform)
  }
  if (t == 0) {
    pl->x = x;
    pl->hi = hi;
    pl->W = W;
    pl->slack = slack[kind];
    pl->range = range;
    pl->few = kind;
    pl->used = used[1];
    pl->total[0] = total[0];
    pl->total[1] = total[1];
    if (blockIdx.x == 0)
      *p.list = SharedList{{total[0], total[1]}, {used[0], used[1]}, W, {slack[0], slack[1]}};
  }
  __syncthreads();
}

// The stretches of a CTA's range, one after another.
struct SharedWalk {
  long long x, hi, first;
  int o, piece0;
  Keys k;
  sh::Shape s;
};
__device__ __forceinline__ void walk_keys(const SharedParams& p, const sh::Plan* pl, SharedWalk& w) {
  if (w.o < sh::KEPT) {
    w.k.lo = pl->lo[w.o];
    w.k.hi = pl->end[w.o];
    w.k.tab = pl->tab[w.o];
    const bool seq = w.o >= p.groups;
    w.k.row0 = seq ? w.o - p.groups : (w.o < pl->groups ? pl->starts[w.o] : 0);
    w.k.rows = seq ? p.SqG : (w.o < pl->groups ? (pl->starts[w.o + 1] - pl->starts[w.o]) * p.SqG : 0);
  } else {
    w.k = keys_of(p, pl, w.o);
  }
}
__device__ __forceinline__ void walk_owner(const SharedParams& p, const sh::Plan* pl, SharedWalk& w) {
  walk_keys(p, pl, w);
  w.s = shape_of(p, pl->few, w.k.rows, w.k.lo, w.k.hi, pl->W);
}
__device__ __forceinline__ SharedWalk walk_start(const SharedParams& p, const sh::Plan* pl) {
  SharedWalk w = {};
  w.o = pl->o;
  if (w.o < 0) return w;  // (x = hi: no stretch)
  w.x = pl->x;
  w.hi = pl->hi;
  w.first = pl->first;
  w.piece0 = pl->piece0;
  walk_keys(p, pl, w);
  w.s = pl->s;
  return w;
}
__device__ __forceinline__ bool walk_next(const SharedParams& p, const sh::Plan* pl, SharedWalk& w,
                                          int range, sh::Seg* g) {
  int s, rt, at, n;
  for (;;) {
    if (w.x >= w.hi) return false;
    long long per = places_per_head(w.s, pl->slack);
    while (w.x >= w.first + per * p.Hkv) {
      w.first += per * p.Hkv;
      w.piece0 += (int)pieces_of(p, w.s);
      if (++w.o >= p.groups + p.B) return false;  // (the range ends at the list's end)
      if (w.o == p.groups) w.piece0 = 0;
      walk_owner(p, pl, w);
      per = places_per_head(w.s, pl->slack);
    }
    long long y = w.x - w.first;
    g->hkv = (int)quotient(y, per);
    y -= g->hkv * per;
    const long long strip = (long long)w.s.n_rt * ((long long)w.s.len * w.s.cost + pl->slack);
    s = (int)quotient(y, strip);
    y -= s * strip;
    const int len = min(w.s.len, w.s.T - s * w.s.len);
    const long long piece = (long long)len * w.s.cost + pl->slack;
    rt = (int)quotient(y, piece);
    y -= rt * piece;
    // Tiles whose first place lies in the range.
    const long long begin = w.x - y;
    at = (int)quotient(y + w.s.cost - 1, w.s.cost);
    if (at < len) {
      const long long end = quotient(w.hi - begin + w.s.cost - 1, w.s.cost);
      n = (int)(end < len ? end : len) - at;
      w.x = begin + (long long)(at + n) * w.s.cost;
      if (n <= 0) return false;
      break;
    }
    w.x = begin + piece;  // slack
  }
  g->kind = w.o < p.groups ? 0 : 1;
  g->r0 = rt * 2 * sh::BM;
  g->rows = min(2 * sh::BM, w.k.rows - g->r0);
  g->t = w.s.t0 + s * w.s.len + at;
  g->n = n;
  // Stretches in list order: each begins a piece or a CTA's range.
  g->id = w.piece0 + (g->hkv * w.s.S + s) * w.s.n_rt + rt + range;
  g->lo = w.k.lo;
  g->hi = w.k.hi;
  g->row0 = w.k.row0;
  g->tab = w.k.tab;
  g->twice = w.s.n_rt > 1;
  return true;
}

// Query row r of a unit: its index in [B, Sq, Hq], and its new token.
__device__ __forceinline__ size_t shared_qrow(const SharedParams& p, int row0, int hkv, int r,
                                              int* s_out) {
  const int m = r / p.SqG, e = r - m * p.SqG, s = e / p.G;
  *s_out = s;
  return ((size_t)(row0 + m) * p.Sq + s) * p.Hq + (size_t)hkv * p.G + (e - s * p.G);
}

// The MMAs' steps of 16 along the contracted axis.  Addresses in units of 16 bytes.
// D (tensor memory at d) = A B^T, both with D elements per row in 128-byte rows, half
// after half (A's halves HALF_BYTES apart).
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b, uint32_t b_half,
                                           uint32_t hi, uint32_t idesc) {
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
    mma_ss_lh(d, a + (((k >> 2) * sh::HALF_BYTES + (k & 3) * 32) >> 4), hi,
              b + (k >> 2) * b_half + (k & 3) * 2, hi, idesc, k > 0 ? 1u : 0u);
}
// (+)= P (tensor memory) V.
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t p, uint32_t v, uint32_t hi,
                                           uint32_t idesc, bool add) {
#pragma unroll
  for (int k = 0; k < sh::BN / 16; ++k)
    mma_ts_lh(d, p + k * 8, v + (uint32_t)((k * 16 * 128) >> 4), hi, idesc,
              add || k > 0 ? 1u : 0u);
}
// A warp's rows (up to 8 NB, as the MMAs' N) against its stretch of keys.  Lane (g, tq)
// = (lane / 4, lane % 4) holds, of row block nb, rows 8 nb + 2 tq + {0, 1}, and of O^T
// the elements 16 dm + g (+ 8).
template <int D, int NB>
struct StreamRows {
  uint32_t q[NB][D / 16][2];
  float m[NB][2], l[NB][2], acc[NB][D / 16][4];
};
template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    mma_fp16_16816(d, a, b0, b1);
  else
    mma_bf16_16816(d, a, b0, b1);
}
// One tile of 32 keys: S^T = K Q^T (A = K rows by ldmatrix, B = Q from registers), an
// online softmax, O^T += V^T P^T (A = V by transposing ldmatrix, B = P^T, the scores'
// accumulator transposed per 8 x 8).  Keys [from, to) of the tile count; lim: of them the
// rows' own limits.  (P is rounded to the inputs' type, as in the tiles of many rows.)
template <int D, int NB, typename T>
__device__ __forceinline__ void stream_tile(StreamRows<D, NB>& w, uint32_t k_tile, uint32_t v_tile,
                                            float c, bool masked, int from, int to,
                                            const int (&lim)[NB][2]) {
  constexpr int MB = sh::FEW_KEYS / 16, HALF = sh::FEW_KEYS * 128;
  constexpr float NEG_INF = -INFINITY;
  const int lane = threadIdx.x & 31, g = lane >> 2, mi = lane >> 3;
  float sc[NB][MB][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) sc[nb][mb][0] = sc[nb][mb][1] = sc[nb][mb][2] = sc[nb][mb][3] = 0.f;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {  // (independent sums side by side)
      const int tok = mb * 16 + (mi & 1) * 8 + (lane & 7), chunk = kk * 2 + (mi >> 1);
      uint32_t a[4];
      ldsm_x4(k_tile + (chunk >> 3) * HALF + tok * 128 + (((chunk & 7) ^ (tok & 7)) << 4), a[0], a[1],
              a[2], a[3]);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma_16816<T>(sc[nb][mb], a, w.q[nb][kk][0], w.q[nb][kk][1]);
    }
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tl = mb * 16 + g + (i >> 1) * 8;
        sc[nb][mb][i] *= c;
        if (masked && (tl < from || tl >= to || tl >= lim[nb][i & 1])) sc[nb][mb][i] = NEG_INF;
      }
  uint32_t pb[NB][MB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float f[2], base[2], rs[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float mx = NEG_INF;
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) mx = fmaxf(mx, fmaxf(sc[nb][mb][e], sc[nb][mb][2 + e]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float top = fmaxf(w.m[nb][e], mx);
      base[e] = top == NEG_INF ? 0.f : top;
      f[e] = fast_exp2(w.m[nb][e] - base[e]);
      w.m[nb][e] = top;
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sc[nb][mb][i] = fast_exp2(sc[nb][mb][i] - base[i & 1]);
        rs[i & 1] += sc[nb][mb][i];
      }
      pb[nb][mb][0] = movmatrix_trans(TileType<T>::pack(sc[nb][mb][0], sc[nb][mb][1]));
      pb[nb][mb][1] = movmatrix_trans(TileType<T>::pack(sc[nb][mb][2], sc[nb][mb][3]));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) w.l[nb][e] = w.l[nb][e] * f[e] + rs[e];
    // (Mostly no row has a new maximum: the products stay as they are.)
    if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
      for (int dm = 0; dm < D / 16; ++dm) {
        w.acc[nb][dm][0] *= f[0];
        w.acc[nb][dm][1] *= f[1];
        w.acc[nb][dm][2] *= f[0];
        w.acc[nb][dm][3] *= f[1];
      }
    }
  }
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int dm = 0; dm < D / 16; ++dm) {
      const int tok = mb * 16 + (mi >> 1) * 8 + (lane & 7), chunk = dm * 2 + (mi & 1);
      uint32_t a[4];
      ldsm_x4_t(v_tile + (chunk >> 3) * HALF + tok * 128 + (((chunk & 7) ^ (tok & 7)) << 4), a[0], a[1],
                a[2], a[3]);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma_16816<T>(w.acc[nb][dm], a, pb[nb][mb][0], pb[nb][mb][1]);
    }
}

// A streaming warp's walk, in shared memory (its registers hold its rows): the walk, and
// the stretches begun, of which the loads are two tiles ahead of the arithmetic.
struct StreamWalk {
  SharedWalk w;
  sh::Seg told[4];
};
static_assert(sizeof(StreamWalk) <= 288, "a streaming warp's walk");

// One warp's range of the sequences' list, from its loads to its partials.  tiles: two
// of K and V each; full: their barriers.  The loads run two tiles ahead of the
// arithmetic, over the ends of stretches.
template <int D, typename T, int NB>
__device__ __forceinline__ void stream_keys(const SharedParams& p, const sh::Plan* pl,
                                            const CUtensorMap* tmK, const CUtensorMap* tmV,
                                            uint8_t* tiles, uint64_t* full, StreamWalk* sw, int warp,
                                            volatile int* abort_flag) {
  using C = sh::Cfg<D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int range = pl->range + warp;
  if (range >= pl->used || pl->o < 0) return;
  if (lane == 0) {
    sw->w = walk_start(p, pl);
    sw->w.x = pl->total[0] + quotient(pl->total[1] * range, pl->used);
    sw->w.hi = pl->total[0] + quotient(pl->total[1] * (range + 1), pl->used);
  }
  const uint64_t pol = l2_policy_evict_first();
  // The loading side: the next tile of its stretch and that one's tiles, 32 pages of the row.
  int ld_at = 0, ld_n = 0, ld_tab = -1, ids_base = 0, ids = -1;
  bool ld_more = true;
  uint32_t loaded = 0, used = 0, seg_ld = 0, seg = 0;  // tiles, stretches begun
  uint32_t bad_bits = 0;  // of the tile in either buffer: it has no page
  // The side that computes: the next tile of its stretch, its rows.
  int at = 0;
  StreamRows<D, NB> r;
  int lim0[NB][2];
  bool ok = true;
  for (;;) {
    while (ld_more && loaded - used < 2) {
      if (ld_at == ld_n) {
        ld_at = 0;
        if (lane == 0) {
          sh::Seg next;
          if (!walk_next(p, pl, sw->w, range, &next)) next.kind = -1;
          sw->told[seg_ld & 3] = next;
        }
        __syncwarp();
        if (!(ld_more = sw->told[seg_ld & 3].kind >= 0)) break;
        ld_n = sw->told[seg_ld & 3].n;
        ++seg_ld;
      }
      const sh::Seg& ld = sw->told[(seg_ld - 1) & 3];
      const int buf = loaded & 1;
      const int key = (ld.t + ld_at) * sh::FEW_KEYS, page = key / p.page_size;
      const int row = key - page * p.page_size;
      if (ld.tab != ld_tab || page < ids_base || page >= ids_base + 32) {
        ld_tab = ld.tab;
        ids_base = page;
        ids = page + lane < p.max_pages
                  ? p.page_table[(size_t)ld.tab * p.max_pages + page + lane]
                  : -1;
      }
      const int id = __shfl_sync(0xffffffffu, ids, page - ids_base);
      const bool bad = id < 0 || id >= p.num_pages;
      bad_bits = (bad_bits & ~(1u << buf)) | (uint32_t)bad << buf;
      if (lane == 0) {
        if (bad) {
          atomicOr(&g_shared_err, kErrBounds);
          mbar_arrive(&full[buf]);
        } else {
          mbar_arrive_expect_tx(&full[buf], 2 * C::FEW_KV);
#pragma unroll
          for (int h = 0; h < C::HALVES; ++h) {
            uint8_t* const dst = tiles + buf * 2 * C::FEW_KV + h * C::FEW_HALF;
            tma_load_4d_hint(dst, tmK, &full[buf], h * 64, ld.hkv, row, id, pol);
            tma_load_4d_hint(dst + C::FEW_KV, tmV, &full[buf], h * 64, ld.hkv, row, id, pol);
          }
        }
      }
      __syncwarp();
      ++loaded;
      ++ld_at;
    }
    if (used == loaded) break;
    if (at == 0) ++seg;
    const sh::Seg& sg = sw->told[(seg - 1) & 3];
    if (at == 0) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        int s;
        const int row = nb * 8 + g;
        const bool real = row < p.SqG;
        const uint32_t* const src = reinterpret_cast<const uint32_t*>(
            static_cast<const T*>(p.q) + shared_qrow(p, sg.row0, sg.hkv, real ? row : 0, &s) * D);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          r.q[nb][kk][0] = real ? src[kk * 8 + tq] : 0u;
          r.q[nb][kk][1] = real ? src[kk * 8 + 4 + tq] : 0u;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // The row of new token s sees the keys below L - Sq + s + 1.
          const int mine = nb * 8 + 2 * tq + e;
          lim0[nb][e] = sg.hi - p.Sq + 1 + (mine < p.SqG ? mine / p.G : 0);
          r.m[nb][e] = -INFINITY;
          r.l[nb][e] = 0.f;
        }
#pragma unroll
        for (int dm = 0; dm < D / 16; ++dm)
          r.acc[nb][dm][0] = r.acc[nb][dm][1] = r.acc[nb][dm][2] = r.acc[nb][dm][3] = 0.f;
      }
    }
    const int buf = used & 1;
    if (!(ok = mbar_wait<true>(&full[buf], (used >> 1) & 1, abort_flag, &g_shared_err, 16))) break;
    __syncwarp();
    uint8_t* const tile = tiles + buf * 2 * C::FEW_KV;
    const int key0 = (sg.t + at) * sh::FEW_KEYS;
    const int from = bad_bits >> buf & 1 ? sh::FEW_KEYS : max(sg.lo - key0, 0);
    const int to = min(sg.hi - key0, sh::FEW_KEYS);
    const bool masked = from > 0 || key0 + sh::FEW_KEYS > sg.hi - p.Sq + 1;
    if (from > 0 || to < sh::FEW_KEYS) {
      // Rows of keys that nobody sees can hold anything: they are cleared, since 0 *
      // NaN in P V would reach every row.
      for (int x = lane; x < 2 * C::HALVES * sh::FEW_KEYS * 8; x += 32) {
        const int key = x >> 3 & (sh::FEW_KEYS - 1);
        if (key < from || key >= to)
          *reinterpret_cast<uint4*>(tile + x * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      __syncwarp();
    }
    int lim[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) lim[nb][e] = lim0[nb][e] - key0;
    const uint32_t k_tile = smem_u32(tile);
    stream_tile<D, NB, T>(r, k_tile, k_tile + C::FEW_KV, p.c, masked, from, to, lim);
    // The buffer's reads are done before the copy unit writes it again.
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    ++used;
    if (++at < sg.n) continue;
    at = 0;
    // The lanes' parts of each row's sum, and the rows' partials.
    const size_t slot = (size_t)sg.id * p.SqG;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = r.l[nb][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int row = nb * 8 + 2 * tq + e;
        if (row < p.SqG) {
          if (g == 0)
            reinterpret_cast<float2*>(p.part_ml[1])[slot + row] = make_float2(r.m[nb][e], l);
          float* const dst = p.part_o[1] + (slot + row) * D;
#pragma unroll
          for (int dm = 0; dm < D / 16; ++dm) {
            dst[dm * 16 + g] = r.acc[nb][dm][e];
            dst[dm * 16 + g + 8] = r.acc[nb][dm][2 + e];
          }
        }
      }
  }
  // After an abort: the loads that may still be in flight, before shared memory goes.
  if (!ok)
    for (uint32_t u = used; u < loaded; ++u) mbar_wait_drain(&full[u & 1], (u >> 1) & 1);
}

template <int D, typename T>
__global__ void __launch_bounds__(sh::THREADS, 1)
    shared_split_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ CUtensorMap tmK32,
                        const __grid_constant__ CUtensorMap tmV32,
                        const __grid_constant__ SharedParams p) {
  using C = sh::Cfg<D>;
  constexpr int NSTAGE = C::NSTAGE;
  constexpr int W_PROD = 8, W_MMA = 9, W_WALK = 10;
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
  uint64_t* told = drain + 1;       // [RING] a stretch stands in its slot
  uint64_t* heard = told + sh::RING;  // [RING] all warps have read it
  uint64_t* few_full = heard + sh::RING;  // [FEW_WARPS][2] a streaming warp's tiles
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(few_full + 2 * sh::FEW_WARPS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile uint32_t* issued = reinterpret_cast<volatile uint32_t*>(abort_flag + 1);
  volatile uint32_t* tile_bad = issued + 1;  // [BAD_RING]
  static_assert(2 * C::NSTAGE * 8 + (9 + 2 * sh::RING + 2 * sh::FEW_WARPS) * 8 + 12 +
                        4 * sh::BAD_RING <= C::SMEM_BAR, "barrier block");
  uint8_t* const s_ring = reinterpret_cast<uint8_t*>(full) + C::SMEM_BAR;  // stretches told
  sh::Plan* const plan = reinterpret_cast<sh::Plan*>(s_ring + C::SMEM_RING);

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
    for (int i = 0; i < 2 * sh::FEW_WARPS; ++i) mbar_init(&few_full[i], 1);
    for (int i = 0; i < sh::RING; ++i) {
      mbar_init(&told[i], 1);
      mbar_init(&heard[i], 10);  // producer, MMA issuer, eight softmax warps
    }
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

  shared_plan(p, plan);
  if (plan->few) {
    if (warp < sh::FEW_WARPS) {
      uint8_t* const tiles = sQ + warp * 4 * C::FEW_KV;
      if (p.SqG <= 8)
        stream_keys<D, T, 1>(p, plan, &tmK32, &tmV32, tiles, few_full + 2 * warp,
                             reinterpret_cast<StreamWalk*>(s_ring + warp * 288), warp, abort_flag);
      else
        stream_keys<D, T, 2>(p, plan, &tmK32, &tmV32, tiles, few_full + 2 * warp,
                             reinterpret_cast<StreamWalk*>(s_ring + warp * 288), warp, abort_flag);
    }
    __syncthreads();
    if (warp == W_MMA) tmem_dealloc(tmem, C::TMEM_COLS);
    return;
  }
  // The k-th stretch of this CTA; false at the end, and where a wait gave up (*ok).
  uint32_t seg = 0;
  sh::Seg sg;
  auto next_seg = [&](bool* ok) {
    const int slot = seg % sh::RING;
    *ok = mbar_wait<false>(&told[slot], (seg / sh::RING) & 1, abort_flag, &g_shared_err, 13);
    if (!*ok) return false;
    sg = *reinterpret_cast<const sh::Seg*>(s_ring + slot * 64);
    if (warp != W_MMA) __syncwarp();  // (there one lane alone listens)
    if (lane == 0) mbar_arrive(&heard[slot]);
    ++seg;
    return sg.kind >= 0;
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
      while (ok && next_seg(&ok)) {
        const int32_t* table = p.page_table + (size_t)sg.tab * p.max_pages;
        const int end = sg.hi;
        const uint64_t pol = sg.twice ? again : once;
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
        // S[buf] = Q[tile] K^T.
        auto issue_s = [&](int tile, int buf, uint32_t cnt) {
          mma_scores<D>(tmem + C::COL_S + buf * 128, q_lo + tile * (C::TILE_BYTES >> 4),
                        k_lo + (cnt % NSTAGE) * (C::TILE_BYTES >> 4), sh::HALF_BYTES >> 4, sd_hi,
                        IDESC_S);
          mma_commit(&s_full[buf]);
        };
        // O[i] (+)= P[i] V.
        auto issue_pv = [&](int i, uint32_t cnt, bool add) {
          mma_values(tmem + C::COL_O + i * D, tmem + C::COL_S + i * 128,
                     v_lo + (cnt % NSTAGE) * (C::TILE_BYTES >> 4), sd_hi, IDESC_O, add);
        };
        uint32_t tc = 0, cw[2] = {0, 0};
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
        while (ok && next_seg(&ok)) {
          const int n = sg.n;
          if (!(ok = mbar_wait<false>(q_full, (seg - 1) & 1, abort_flag, &g_shared_err, 2))) break;
          tc_fence_after();
          if (!landed(2 * tc, 3)) break;
          if (sg.rows > sh::BM) {  // two row tiles on every key tile
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
    } else if (warp == W_WALK && lane == 0) {
      // ============================ the walk over the range ============================
      SharedWalk w = walk_start(p, plan);
      for (uint32_t k = 0;; ++k) {
        const int slot = k % sh::RING;
        sh::Seg g;
        if (!walk_next(p, plan, w, plan->range, &g)) g.kind = -1;
        if (!mbar_wait<true>(&heard[slot], ((k / sh::RING) & 1) ^ 1, abort_flag, &g_shared_err, 14))
          break;
        *reinterpret_cast<sh::Seg*>(s_ring + slot * 64) = g;
        mbar_arrive(&told[slot]);
        if (g.kind < 0) break;
      }
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
    uint32_t tc = 0, cw = 0, done = 0;
    bool ok = true;
    // This thread's row of Q for a stretch (one row tile: the first warpgroup's).
    auto load_q = [&] {
      const int rr = i * sh::BM + tid;
      if (sg.rows > sh::BM || i == 0) {
        // The warp's 32 rows one after another, a row by D / 8 lanes.
        int s;
        const bool real = rr < sg.rows;
        const int qrow = real ? (int)shared_qrow(p, sg.row0, sg.hkv, sg.r0 + rr, &s) : -1;
        constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;
        const int x = lane % LANES;
        uint4 v[32 / AT_ONCE];
#pragma unroll
        for (int k = 0; k < 32 / AT_ONCE; ++k) {
          const int from = __shfl_sync(0xffffffffu, qrow, k * AT_ONCE + lane / LANES);
          const T* const row = static_cast<const T*>(p.q) + (size_t)max(from, 0) * D;
          v[k] = reinterpret_cast<const uint4*>(row)[x];
          if (from < 0) v[k] = make_uint4(0u, 0u, 0u, 0u);
        }
        uint8_t* const dst = sQ + i * C::TILE_BYTES + (x >> 3) * sh::HALF_BYTES;
#pragma unroll
        for (int k = 0; k < 32 / AT_ONCE; ++k) {
          const int row = wq * 32 + k * AT_ONCE + lane / LANES;
          *reinterpret_cast<uint4*>(dst + row * 128 + (((x & 7) ^ (row & 7)) << 4)) = v[k];
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(q_full);
    };
    bool have = next_seg(&ok);
    if (have) load_q();
    while (have) {
      const int rows = sg.rows, n = sg.n, r0 = sg.r0;
      const bool dual = rows > sh::BM;
      const int kind = sg.kind;
      const int rr = dual ? i * sh::BM + tid : tid;
      const bool row_ok = rr < rows, warp_ok = rr - lane < rows;
      // Keys [lo, end) are somebody's; all rows see those of them below least.
      const int lo = sg.lo, end = sg.hi, t0 = sg.t;
      const int least = kind == 1 ? end - p.Sq + 1 : end;
      const int half = dual ? sh::BM : p.half[kind];
      float* const po = p.part_o[kind] + ((size_t)sg.id * (D / 4) * 2 * p.half[kind] + i * half) * 4;
      float2* const pml = reinterpret_cast<float2*>(p.part_ml[kind]) +
                          (size_t)sg.id * 2 * p.half[kind] + i * half + tid;
      const size_t col = 2 * (size_t)p.half[kind];  // rows of four columns
      // S of the j-th tile is there; V rows that no query sees are cleared (they can hold
      // anything, and 0 * NaN in P V would reach every row).  The tile's first key and
      // missing pages; whether some row does not see all of it.
      int kv0 = 0;
      uint32_t bad = 0;
      bool masked = false;
      auto tile_ready = [&](int j) {
        const uint32_t tj = tc + j;
        ok = mbar_wait<false>(&s_full[i], cw & 1, abort_flag, &g_shared_err, 8 + i);
        if (!ok) return false;
        ++cw;
        __syncwarp();
        tc_fence_after();
        kv0 = (t0 + j) * sh::BN;
        bad = tile_bad[tj % sh::BAD_RING];
        masked = kv0 < lo || kv0 > least - sh::BN || bad;
        if (masked) {
          const Mask128 fine = sound_keys(bad, p.box);
          const uint32_t cv = 2 * tj + 1;
          ok = mbar_wait<false>(&full[cv % NSTAGE], (cv / NSTAGE) & 1, abort_flag, &g_shared_err, 10);
          if (ok)
            clear_rows<D>(sKV + (cv % NSTAGE) * C::TILE_BYTES, wq, lane,
                          Mask128{fine.lo & low_bits(end - kv0) & ~low_bits(lo - kv0),
                                  fine.hi & low_bits(end - kv0 - 64) & ~low_bits(lo - kv0 - 64)});
        }
        return ok;
      };
      // After the last tile: Q of the next stretch, then P V of this one.  False: leave.
      const bool active = dual || i < n;
      auto move_on = [&] {
        tc += n;
        have = false;
        if (ok) have = next_seg(&ok);
        // (seg counts the next stretch by now.)
        if (have) ok = mbar_wait<false>(q_free, seg & 1, abort_flag, &g_shared_err, 11);
        if (!ok) return false;
        if (have) load_q();
        if (!active) return true;
        ok = mbar_wait<false>(&pv_done[i], done & 1, abort_flag, &g_shared_err, 12);
        if (!ok) return false;
        ++done;
        __syncwarp();
        tc_fence_after();
        return true;
      };
      int lim = end;  // this row sees the keys [lo, lim)
      if (kind == 1) {
        int s = 0;
        if (row_ok) shared_qrow(p, 0, 0, r0 + rr, &s);
        lim = least + s;
      }
      float m_used = NEG_INF, l = 0.f;
      for (int j = dual ? 0 : i; j < n; j += dual ? 1 : 2) {
        if (!tile_ready(j)) break;
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
      if (!move_on()) break;
      if (!active) {
        if (row_ok) *pml = make_float2(NEG_INF, 0.f);
        continue;
      }
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
            *reinterpret_cast<float4*>(po + ((q * 8 + x) * col + tid) * 4) =
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

// Merge: a block takes up to merge_rows <= RC rows of one (sequence, kv head) and 256 / RC
// groups of four columns.  A warp for each list finds out where their partials are, of the group's unit and
// of their own (the lanes take strips); then a thread takes four columns of a row and
// walks the lists, 6 or 12 partials' loads at a time.  With fewer rows than RC, the threads of a
// row's columns share the lists.
namespace join {
constexpr int THREADS = 256;
constexpr int resident(int ahead) { return ahead > 6 ? 2 : 4; }  // blocks of an SM
constexpr int LIST = 2048;  // partials of a row from one unit: two per CTA and strip, one per warp
}  // namespace join
template <int D, typename T, int RC, int AHEAD>
__global__ void __launch_bounds__(join::THREADS, join::resident(AHEAD)) shared_merge_kernel(
    const __grid_constant__ SharedParams p) {
  static_assert(RC <= 32, "a row's threads in one warp");
  // Lists: of the group's unit for the rows' first and last pair of row tiles; their own.
  __shared__ int s_list[3][join::LIST];
  __shared__ int s_count[3];
  __shared__ int s_group[2];  // first sequence of the group, or -1; its first such pair
  pdl_launch_dependents();
  const int t = threadIdx.x, lane = t & 31;
  const int chunks = (p.SqG + p.merge_rows - 1) / p.merge_rows, unit = blockIdx.x / chunks;
  const int first = (blockIdx.x - unit * chunks) * p.merge_rows;
  const int rows = min(p.merge_rows, p.SqG - first);
  const int b = unit / p.Hkv, hkv = unit - b * p.Hkv;
  pdl_wait_primary();
  if (t < 96) {  // a warp for each list
    const SharedList list = *p.list;
    const SharedOwner own = p.owner[p.groups + b];
    SharedOwner grp = own;
    if (own.group >= 0) grp = p.owner[own.group];
    const int r0 = (b - grp.row0) * p.SqG + first;  // of the group's unit
    const int l = t >> 5;
    if (t == 0) {
      s_group[0] = own.group >= 0 ? grp.row0 : -1;
      s_group[1] = r0 / (2 * sh::BM);
    }
    if (lane == 0) s_count[l] = 0;
    // The range that holds place y: the largest c with total * c / used <= y.
    auto cta_of = [&](long long y, int k) {
      return (int)quotient((y + 1) * list.used[k] - 1, list.total[k]);
    };
    // (The rows' first and last pair are mostly the same one.)
    if (l == 2 || (own.group >= 0 && (l == 0 || (r0 + rows - 1) / (2 * sh::BM) != r0 / (2 * sh::BM)))) {
      const SharedOwner o = l < 2 ? grp : own;
      const int rt = (l == 0 ? r0 : l == 1 ? r0 + rows - 1 : first) / (2 * sh::BM);
      const int few = p.few && l == 2;
      const sh::Shape s = shape_of(p, few, o.rows, o.lo, o.hi, list.W);
      const int slack = list.slack[few];
      const bool two = few || min(2 * sh::BM, o.rows - rt * 2 * sh::BM) > sh::BM;
      const long long head = o.first + hkv * places_per_head(s, slack);
      int n = 0;
      for (int k0 = 0; s.T > 0 && k0 < s.S; k0 += 32) {
        const int k = k0 + lane;
        int c0 = 0, count = 0;
        if (k < s.S) {
          const int len = min(s.len, s.T - k * s.len);
          const long long piece = (long long)len * s.cost + slack;
          const long long y =
              head + (long long)k * s.n_rt * ((long long)s.len * s.cost + slack) + rt * piece;
          // (A tile belongs to the range that holds its first place.)
          c0 = cta_of(y, few);
          count = (cta_of(y + (long long)(len - 1) * s.cost, few) - c0 + 1) << (two ? 0 : 1);
        }
        int inc = count;
#pragma unroll
        for (int o2 = 1; o2 < 32; o2 <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, inc, o2);
          if (lane >= o2) inc += x;
        }
        // (One row tile: two partials of each CTA, one behind the other.)
        const int id = o.piece0 + (hkv * s.S + k) * s.n_rt + rt + c0;
        for (int e = 0; e < count; ++e) {
          const int at = n + inc - count + e;
          if (at < join::LIST) s_list[l][at] = two ? 2 * (id + e) : 2 * id + e;
        }
        n += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) s_count[l] = min(n, join::LIST);
      if (n > join::LIST && lane == 0) atomicOr(&g_shared_err, kErrBounds);
    }
  }
  __syncthreads();
  int width = 1;  // rows, as a power of two; RC / width threads share a row's list
  while (width < rows) width *= 2;
  const int r = t % width, turn = t / width % (RC / width);
  const int col = blockIdx.y * (join::THREADS / RC) + t / RC;
  const bool real = r < rows;
  const int g_row = s_group[0] < 0 ? 0 : (b - s_group[0]) * p.SqG + first + (real ? r : 0);
  const int l = g_row / (2 * sh::BM) == s_group[1] ? 0 : 1;
  const int n0 = s_group[0] < 0 ? 0 : s_count[l], n = n0 + s_count[2];
  const int at[2] = {g_row % (2 * sh::BM), (first + (real ? r : 0)) % (2 * sh::BM)};
  float M = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto join_in = [&](float2 a, const float4& v) {
    if (!(a.y > 0.f || a.y != a.y)) return;  // saw no key  (NaN joins)
    float wt = 1.f;
    if (a.x > M) {
      const float f = M == -INFINITY ? 0.f : fast_exp2(M - a.x);
      den *= f;
      acc.x *= f;
      acc.y *= f;
      acc.z *= f;
      acc.w *= f;
      M = a.x;
    } else {
      wt = fast_exp2(a.x - M);
    }
    den += wt * a.y;
    acc.x += wt * v.x;
    acc.y += wt * v.y;
    acc.z += wt * v.z;
    acc.w += wt * v.w;
  };
  for (int k = turn; k < n; k += AHEAD * (RC / width)) {
    float2 ml[AHEAD];
    float4 ov[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int item = k + u * (RC / width);
      ml[u] = make_float2(-INFINITY, 0.f);
      if (item < n && real) {
        const int kind = item < n0 ? 0 : 1;
        const int e = kind ? s_list[2][item - n0] : s_list[l][item];
        const bool few = kind && p.few;
        // (Partials of either kind are at most 2^32 times 16 bytes.)
        const uint32_t slots = few ? p.SqG : 2 * p.half[kind];
        const uint32_t slot = at[kind] + (e & 1 ? p.half[kind] : 0), id = e >> 1;
        ml[u] = reinterpret_cast<const float2*>(p.part_ml[kind])[id * slots + slot];
        ov[u] = reinterpret_cast<const float4*>(
            p.part_o[kind])[few ? (id * slots + slot) * (D / 4) + col
                                : (id * (D / 4) + col) * slots + slot];
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) join_in(ml[u], ov[u]);
  }
  for (int o = width; o < RC; o <<= 1) {
    const float2 a =
        make_float2(__shfl_xor_sync(0xffffffffu, M, o), __shfl_xor_sync(0xffffffffu, den, o));
    const float4 v =
        make_float4(__shfl_xor_sync(0xffffffffu, acc.x, o), __shfl_xor_sync(0xffffffffu, acc.y, o),
                    __shfl_xor_sync(0xffffffffu, acc.z, o), __shfl_xor_sync(0xffffffffu, acc.w, o));
    join_in(a, v);
  }
  if (!real || turn != 0) return;
  const int own_r = first + r, tok = own_r / p.G;
  const size_t row = ((size_t)b * p.Sq + tok) * p.Hq + (size_t)hkv * p.G + (own_r - tok * p.G);
  const float inv = den == 0.f ? 0.f : 1.f / den;
  *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + row * D + col * 4) = make_uint2(
      TileType<T>::pack(acc.x * inv, acc.y * inv), TileType<T>::pack(acc.z * inv, acc.w * inv));
  if (p.lse && col == 0)
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
static cudaError_t launch_shared(SharedParams& p, const CUtensorMap (&tm)[4],
                                 cudaStream_t stream) {
  using C = sh::Cfg<D>;
  constexpr int ALL = join::THREADS * 4 / D;  // rows of a merge block that takes all columns
  static int attr_set[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !__atomic_load_n(&attr_set[dev], __ATOMIC_ACQUIRE)) {
    e = cudaFuncSetAttribute(shared_split_kernel<D, T>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_TOTAL);
    if (e != cudaSuccess) return e;
    // As in the tree decode: the merge keeps the split kernel's division of the SM.
    for (auto k : {shared_merge_kernel<D, T, ALL, 6>, shared_merge_kernel<D, T, 32, 6>,
                   shared_merge_kernel<D, T, 32, 12>}) {
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
  e = cudaLaunchKernelEx(&cfg, shared_split_kernel<D, T>, tm[0], tm[1], tm[2], tm[3], p);
  if (e != cudaSuccess) return e;
  // Blocks of 32 rows' threads while all of them are resident at once: a row then has more
  // of them (48 sequences of 16 rows, D = 64: 30.6 us, 34.9 with blocks of all columns; 8 of
  // 4 rows and 8200 keys 24.0, 26.0 with 6 loads at a time; 64 of 8 rows, whose blocks are
  // not all resident, 69 us, 61 with blocks of all columns).
  // (And fewer rows to a block as long as they are: 3 sequences of 32 rows behind 44000
  // keys, D = 64, 34 us instead of 90.)
  const long long units = (long long)p.B * p.Hkv;
  auto blocks = [&](int rows) { return units * ((p.SqG + rows - 1) / rows); };
  auto fits = [&](int rows, int ahead) {
    return blocks(rows) * (D / 32) <= (long long)join::resident(ahead) * p.ctas;
  };
  for (int rows = 1; rows <= 32; rows *= 2) {
    p.merge_rows = rows;
    const dim3 grid((unsigned)blocks(rows), D / 32);
    if (fits(rows, 12))
      return launch_dependent(shared_merge_kernel<D, T, 32, 12>, grid, join::THREADS, stream, p);
    if (rows == 32 && fits(rows, 6))
      return launch_dependent(shared_merge_kernel<D, T, 32, 6>, grid, join::THREADS, stream, p);
  }
  p.merge_rows = ALL;
  return launch_dependent(shared_merge_kernel<D, T, ALL, 6>, dim3((unsigned)blocks(ALL)),
                          join::THREADS, stream, p);
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
  p.few = p.SqG <= fa::sh::FEW;
  p.share_few = fa::sh::share_few(p.SqG, D);
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  // Keys per TMA box: a tile's boxes must not straddle pages.
  p.box = page_size % 128 == 0 ? 128 : (page_size % 64 == 0 ? 64 : 32);
  p.c = scale * 1.4426950408889634f;
  // scale == 0: every visible score is 0; a tiny c keeps hidden keys at -inf.
  if (p.c == 0.f) p.c = 1e-30f;
  p.keep_tiles = fa::sh::L2_KEEPS / (2 * fa::sh::BN * 2 * D);
  p.ctas = fa::sm_count() > 0 ? fa::sm_count() : 148;
  if (p.ctas > fa::join::LIST / 8) p.ctas = fa::join::LIST / 8;
  // Slots: every piece, and one more for each boundary between CTAs' ranges.  Pieces:
  // one per (row-tile pair, kv head), and strips, of which all have at most one per CTA
  // beyond those.
  const long long rows_all = (long long)B * p.SqG, pair = 2 * fa::sh::BM;
  const long long units[2] = {
      groups > 0 ? (groups < B / 2 ? groups : B / 2) + rows_all / pair : 0,
      (long long)B * ((p.SqG + pair - 1) / pair)};
  size_t slots[2], bytes = 0, at_o[2], at_ml[2];
  const size_t owners = (size_t)groups + B;
  bytes = owners * sizeof(fa::SharedOwner) + sizeof(fa::SharedList);
  bytes = (bytes + 255) / 256 * 256;
  for (int k = 0; k < 2; ++k) {
    const long long rows = k == 0 ? rows_all : p.SqG;
    p.half[k] = (int)(rows < fa::sh::BM ? rows : fa::sh::BM);
    const bool few = k == 1 && p.few;
    slots[k] = k == 0 && groups == 0
                   ? 0
                   : (size_t)units[k] * Hkv + (few ? fa::sh::FEW_WARPS : 2) * (size_t)p.ctas;
    const size_t in_slot = few ? p.SqG : 2 * p.half[k];
    // The merge counts 16-byte pieces of partials in 32 bits.
    if (slots[k] * in_slot * (D / 4) > (size_t)1 << 32) return FA_ERR_UNSUPPORTED;
    at_o[k] = bytes;
    bytes += slots[k] * D * in_slot * sizeof(float);
    at_ml[k] = bytes;
    bytes += slots[k] * 2 * in_slot * sizeof(float);
    bytes = (bytes + 255) / 256 * 256;
  }
  CUtensorMap tm[4];
  if (fa::encode_tmap_rows(&tm[0], kpages, D, Hkv, page_size, num_pages, p.box) ||
      fa::encode_tmap_rows(&tm[1], vpages, D, Hkv, page_size, num_pages, p.box) ||
      fa::encode_tmap_rows(&tm[2], kpages, D, Hkv, page_size, num_pages, fa::sh::FEW_KEYS) ||
      fa::encode_tmap_rows(&tm[3], vpages, D, Hkv, page_size, num_pages, fa::sh::FEW_KEYS))
    return fa::record_cuda_status(cudaErrorInvalidValue, "shared decode tensor maps");
  void* scratch = nullptr;
  cudaError_t e = fa::scratch_alloc(&scratch, bytes, stream);
  if (e != cudaSuccess) return fa::record_cuda_status(e, "shared decode scratch");
  uint8_t* const base = static_cast<uint8_t*>(scratch);
  p.owner = reinterpret_cast<fa::SharedOwner*>(base);
  p.list = reinterpret_cast<fa::SharedList*>(base + owners * sizeof(fa::SharedOwner));
  for (int k = 0; k < 2; ++k) {
    p.part_o[k] = reinterpret_cast<float*>(base + at_o[k]);
    p.part_ml[k] = reinterpret_cast<float*>(base + at_ml[k]);
  }
  const bool bf16 = dtype == FA_BF16;
  if (D == 64)
    e = bf16 ? fa::launch_shared<64, __nv_bfloat16>(p, tm, stream)
             : fa::launch_shared<64, __half>(p, tm, stream);
  else
    e = bf16 ? fa::launch_shared<128, __nv_bfloat16>(p, tm, stream)
             : fa::launch_shared<128, __half>(p, tm, stream);
  const cudaError_t ef = cudaFreeAsync(scratch, stream);
  if (e != cudaSuccess) return fa::record_cuda_status(e, "shared decode launch");
  return fa::record_cuda_status(ef, "shared decode cudaFreeAsync");
}
