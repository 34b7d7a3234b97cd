// Steps of the query-row tiles of a chunk, and their sums, in closed form.
//
// A request of n cached rows, the last c of them new, with H heads: its c * H
// query rows (token by token) go in tiles of 128; a tile walks the keys that
// its last token sees, 256 per step.  Tile t's last row 128 t + 127 is one of
// token (128 t + 127) / H, which sees n - c + that + 1 keys, so with floors
// throughout
//     steps(t) = (n - c + (128 t + 127) / H + 256) / 256
//              = (128 t + 127 + (n - c + 256) H) / (256 H) = (t + u) / (2 H),
//     u = (127 + (n - c + 256) H) / 128,
// which is too much for the request's last tile alone: that takes the steps of
// all n keys.  Sums over t of such quotients are those of whole runs of 2 H
// equal ones and a part of a run: no tile is ever listed.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MLAV_HD __host__ __device__ __forceinline__
#else
#define MLAV_HD inline
#endif

namespace mlav {

struct ChunkSteps {
  long long m, u, tiles, last;   // last: steps of the last tile
  int unit, per_tile;            // what a step costs, and a tile beside its steps

  MLAV_HD ChunkSteps(int n, int c, int H, int step_cost, int tile_cost)
      : m(2LL * H), u((127 + (static_cast<long long>(n) - c + 256) * H) / 128),
        tiles((static_cast<long long>(c) * H + 127) / 128), last((static_cast<long long>(n) + 255) / 256), unit(step_cost),
        per_tile(tile_cost) {}
  MLAV_HD long long steps(long long t) const { return t + 1 < tiles ? divide(t + u, m) : last; }
  // (A 64-bit division takes several times as long as a 32-bit one.)
  static MLAV_HD long long divide(long long x, long long by) {
    return x >> 32 ? x / by : static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(by));
  }
  // Sum of y / m over 0 <= y < x.
  MLAV_HD long long quotients(long long x) const {
    const long long q = divide(x, m), r = x - q * m;
    return m * (q * (q - 1) / 2) + r * q;
  }
  // Cost of the first t tiles (t <= tiles).
  MLAV_HD long long before(long long t) const {
    if (t <= 0) return 0;
    const long long whole = t < tiles ? t : tiles - 1;
    return unit * (quotients(whole + u) - quotients(u) + (t < tiles ? 0 : last)) + per_tile * t;
  }
  MLAV_HD long long total() const { return before(tiles); }
  // The tile in which cost x lies, 0 <= x < total().
  MLAV_HD long long tile_at(long long x) const {
    long long lo = 0, hi = tiles;
    while (hi - lo > 1) {
      const long long mid = (lo + hi) / 2;
      if (before(mid) <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  }
};

}  // namespace mlav
