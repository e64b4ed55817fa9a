// fa_shares.h -- how the shared decode's CTAs are shared out between its two lists: tiles of
// units of many rows, and keys that warps stream.  Plain integer arithmetic, the same on the
// device and the host.
#pragma once

#ifdef __CUDACC__
#define FA_BOTH __host__ __device__ __forceinline__
#else
#define FA_BOTH inline
#endif

namespace fa {

// a / b in 32 bits where both fit (not negative).
FA_BOTH long long quotient(long long a, long long b) {
  return (a | b) >> 32 == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

namespace sh {
// What a place costs in time, for the sharing out of the CTAs: 16 in the list of tiles, and
// in the streamed one 5 up to 8 rows, up to 16 rows 10 (D = 128) or 6 (D = 64).  Measured: 64
// sequences of 8 rows behind 8192 keys 75, 58.5, 60, 66 us at 2, 4, 5, 6, behind 32768 114 and
// 99 at 4 and 5; 32 of 16 rows (D = 128) 194, 163, 146 at 6, 8, 10; 48 of 16 rows and 2000 keys
// (D = 64) 37, 41, 43 at 6, 8, 10.
constexpr int SHARE_MANY = 16;
constexpr int share_few(int rows, int D) { return rows <= 8 ? 5 : (D == 128 ? 10 : 6); }

// CTAs of `ctas` (two or more) for the list of tiles: all or none where the other list or this
// one is empty, else one of each kind at least.  starts: places that the streamed list's units
// cost beside those that it has.
FA_BOTH int ctas_of_tiles(long long tiles, long long streamed, long long starts, int ctas,
                          int cost_few) {
  if (tiles == 0) return 0;
  if (streamed == 0) return ctas;
  const long long many = tiles * SHARE_MANY, few = (streamed + starts) * cost_few;
  const long long x = quotient(many * ctas, many + few);
  return x < 1 ? 1 : (x > ctas - 1 ? ctas - 1 : (int)x);
}
}  // namespace sh
}  // namespace fa
