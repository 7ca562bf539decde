// Host-only driver for tests/test_kv_rows.py: the positions that rows of a
// sequence see, by the functions that the attention kernels use and by 64-bit
// arithmetic, over the ends of their ranges.  Prints the number of
// comparisons; exits with 1 at the first difference.  (Built with checks of
// signed overflow.)  No CUDA call is made.
#include <climits>
#include <cstdio>

#include "sgr_kv_attn.cuh"

int main() {
  const int lens[] = {0, 1, 2, 63, 200, 1 << 20, INT_MAX - 127};
  const int rows[] = {1, 2, 3, 64, 201, 1 << 20};
  const int windows[] = {1, 2, 63, 1 << 20, INT_MAX - 1, INT_MAX};
  long long count = 0;
  for (int len : lens)
    for (int n : rows)
      for (int tok : {0, 1, n / 2, n - 2, n - 1}) {
        if (tok < 0 || tok >= n) continue;
        const long long pos = (long long)len - n + tok;
        const int last = sgr::row_last(len - n, tok);
        for (int window : windows)
          for (long long at : {0LL, 1LL, pos - window, pos - window + 1, pos - 1, pos, pos + 1, (long long)len - 1}) {
            if (at < 0 || at >= INT_MAX) continue;
            const bool want = pos >= 0 && at <= pos && at > pos - window;
            const bool span = at >= sgr::row_first(0, last, window) && at <= last;
            ++count;
            if (sgr::row_sees((int)at, last, window) != want || span != want) {
              std::printf("len %d rows %d row %d window %d position %lld\n", len, n, tok, window, at);
              return 1;
            }
          }
      }
  std::printf("%lld\n", count);
  return 0;
}
