// How the tiles of attention with few rows are cut (attend_piece_tiles), over totals up to
// what a call may have: the pieces cover them, none is longer than an even cut and the limit
// on a unit's parts ask for, and a unit lies in as many pieces as the join takes.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "nvfp4_plan.hpp"

int main() {
  using namespace nvfp4;
  const int64_t most = (int64_t(1) << 31) - 1;
  long checked = 0;
  for (int64_t pieces : {int64_t(4), int64_t(8), int64_t(100), int64_t(1024), 4 * kAttendPieces})
    for (int64_t total = 1; total <= most; total = total < 3000 ? total + 1 : total < most ? (total * 9 / 8 < most ? total * 9 / 8 : most) : most + 1)
      for (int64_t near = -3; near <= 0; ++near) {
        const int64_t t = total + near * 700;
        if (t < 1) continue;
        for (int64_t longest : {int64_t(1), t < 513 ? t : int64_t(513), t < (1 << 24) ? t : int64_t(1) << 24}) {
          const int64_t per = attend_piece_tiles(t, longest, pieces);
          const bool covers = per >= 1 && per * pieces >= t;
          const bool even = (per - 1) * pieces < t || (per - 1) * kMostParts < longest;
          const bool parts = (longest + per - 1) / per <= kMostParts;
          ++checked;
          if (!covers || !even || !parts || per > most) {
            printf("total %lld longest %lld pieces %lld: %lld tiles a piece\n", (long long)t, (long long)longest, (long long)pieces, (long long)per);
            return 1;
          }
        }
      }
  printf("%ld cuts\n", checked);
  return 0;
}
