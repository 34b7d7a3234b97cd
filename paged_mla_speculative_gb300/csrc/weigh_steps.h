// Steps of a request whose rows are weighed, and their sums, in closed form.
//
// A request of n cached rows, the last c of them new, with H heads: keys go in
// blocks of 256, the c * H query rows (token by token) in tiles of 256; a step
// is one tile against one block, block by block.  Key j is seen by token i >=
// j - (n - c), so block kb starts with tile
//     first(kb) = max(0, floor((256 kb - (n - c)) H / 256)) = max(0, kb H - A),
//     A = ceil((n - c) H / 256),
// and the steps before a block are a sum over an arithmetic run.
#pragma once

#include <stdint.h>

#include "chunk_steps.h"   // MLAV_HD

namespace mlav {

struct WeighSteps {
  long long H, A, k0, tiles, blocks;   // first(k0) is 0, first(k0 + 1) is not

  MLAV_HD WeighSteps() : H(1), A(0), k0(0), tiles(0), blocks(0) {}
  MLAV_HD WeighSteps(int n, int c, int heads)
      : H(heads), A(((static_cast<long long>(n) - c) * heads + 255) / 256), k0(A / heads),
        tiles((static_cast<long long>(c) * heads + 255) / 256), blocks(c > 0 ? (static_cast<long long>(n) + 255) / 256 : 0) {}
  MLAV_HD long long first(long long kb) const { return kb * H > A ? kb * H - A : 0; }
  // Steps of the blocks before kb.
  MLAV_HD long long before(long long kb) const {
    const long long m = kb - 1;
    const long long skipped = m > k0 ? H * (m * (m + 1) / 2 - k0 * (k0 + 1) / 2) - A * (m - k0) : 0;
    return kb * tiles - skipped;
  }
  MLAV_HD long long total() const { return before(blocks); }
  // The block of step x, 0 <= x < total().
  MLAV_HD long long block_at(long long x) const {
    long long lo = 0, hi = blocks;
    while (hi - lo > 1) {
      const long long mid = (lo + hi) / 2;
      if (before(mid) <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  }
};

}  // namespace mlav
