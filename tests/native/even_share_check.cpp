// Host-only check of the deal of items to blocks (compiled with g++ by
// tests/test_even_share_cpu.py): every item in one share, in order, none empty
// while another has two more, up to the most items an int counts.
#include <cstdint>
#include <cstdio>

#include "even_share.h"

int main() {
  const int sizes[] = {0, 1, 7, 151, 152, 153, 1000, 28256364, 28256365, 33554432, 134217720,
                       INT32_MAX};
  const int grids[] = {1, 2, 3, 76, 151, 152};
  for (const int items : sizes)
    for (const int blocks : grids) {
      int at = 0, least = INT32_MAX, most = 0;
      for (int b = 0; b < blocks; ++b) {
        const mxfp8::EvenShare s = mxfp8::even_share(items, b, blocks);
        const int n = s.last - s.first;
        if (s.first != at || n < 0) {
          std::printf("FAIL %d items, block %d of %d: %d..%d after %d\n", items, b, blocks, s.first,
                      s.last, at);
          return 1;
        }
        at = s.last;
        least = n < least ? n : least;
        most = n > most ? n : most;
      }
      if (at != items || most - least > 1) {
        std::printf("FAIL %d items, %d blocks: end %d, %d to %d each\n", items, blocks, at, least,
                    most);
        return 1;
      }
    }
  std::printf("ok\n");
  return 0;
}
