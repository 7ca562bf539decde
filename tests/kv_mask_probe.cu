// Host-only driver for tests/test_kv_mask_host.py: what rows see under windows,
// sinks and trees, by the functions that the kernels use and position by position
// in 64-bit arithmetic, at the ends of their ranges too.  Prints the number of
// comparisons; exits with 1 at the first difference.  (Built with checks of signed
// overflow.)  No CUDA call is made.
#include <climits>
#include <cstdio>
#include <vector>

#include "sgr_kv_mass.cuh"

namespace {

long long count = 0;

bool fail(const char* what, long long a, long long b, long long c, long long d) {
  std::printf("%s: %lld %lld %lld %lld\n", what, a, b, c, d);
  return false;
}

// row_sees, row_bits and mass_rows of every row of a sequence.
bool masks(int len, int n, int group, int window, int sinks, const std::vector<unsigned long long>* tree, int words) {
  sgr::AttnParams p = {};
  p.window = window;
  p.sinks = sinks;
  p.group = group;
  p.tree = tree ? tree->data() : nullptr;
  p.tree_words = words;
  p.tree_stride = words;
  const int first = len - n;
  for (int tok = 0; tok < n; ++tok) {
    const long long place = (long long)first + tok;
    int last = sgr::row_last(first, tok);
    if (tree) {
      const sgr::TreeRow r = sgr::tree_row(p, 0, n, first, tok);
      int bits = 0;
      for (int j = 0; j < n; ++j)
        bits += place >= 0 && (long long)first + j >= 0 && j < 64 * words && ((*tree)[tok * words + j / 64] >> (j % 64) & 1) ? 1 : 0;
      const int want = place < 0 ? -1 : (first > 0 ? first : 0) + (bits > 1 ? bits - 1 : 0);
      if (r.last != want || (place >= 0 && r.drafts != (bits > 0))) return fail("tree row", tok, r.last, want, bits);
      last = r.last;
    }
    const int from = len > 700 ? len - 700 : 0;
    for (int x = from / 32 * 32; x >= 0 && x < len; x = x > INT_MAX - 32 ? -1 : x + 32) {
      const uint32_t got = sgr::row_bits(p, x, last, len, first, tok);
      for (int e = 0; e < 32 && (long long)x + e < len; ++e) {
        const long long t = (long long)x + e;
        bool want = place >= 0 && t <= last && (t > (long long)last - window || t < sinks);
        if (tree && t >= first) {
          const long long j = t - first;
          want = place >= 0 && j < 64LL * words && ((*tree)[tok * words + j / 64] >> (j % 64) & 1);
        }
        ++count;
        if ((got >> e & 1) != (want ? 1u : 0u)) return fail("row bits", len, tok, t, want);
        if (tree) continue;
        if (sgr::row_sees((int)t, last, window, sinks) != want) return fail("row sees", len, tok, t, want);
        for (int g : {0, group - 1}) {  // the row among 32 columns from r on
          const int row = tok * group + g, r = row / 32 * 32;
          const uint32_t rows = sgr::mass_rows(p, (int)t, first, r, n * group);
          if ((rows >> (row - r) & 1) != (want ? 1u : 0u)) return fail("rows", len, row, t, want);
        }
      }
    }
  }
  return true;
}

}  // namespace

int main() {
  for (int len : {0, 1, 31, 200, 1000, INT_MAX - 127})
    for (int n : {1, 3, 33, 70})
      for (int group : {1, 5})
        for (int window : {1, 2, 100, INT_MAX - 1, INT_MAX})
          for (int sinks : {0, 1, 40, 500, INT_MAX})
            if (!masks(len, n, group, window, sinks, nullptr, 0)) return 1;
  unsigned long long seed = 88172645463325252ULL;
  auto random = [&] { return seed ^= seed << 13, seed ^= seed >> 7, seed ^= seed << 17; };
  for (int len : {0, 1, 31, 200, 1000, INT_MAX - 127})
    for (int n : {1, 20, 64, 65, 150})
      for (int words : {1, 2, 3})
        for (int window : {1, 30, INT_MAX})
          for (int sinks : {0, 40}) {
            std::vector<unsigned long long> tree(n * words);
            for (auto& w : tree) w = random() & random();
            if (!masks(len, n, 1, window, sinks, &tree, words)) return 1;
          }
  // Tiles of the sinks come right before the window's.
  for (int tlo : {0, 1, 127, 128, 1000, INT_MAX - 128})
    for (int sinks : {0, 1, 128, 129, 5000, INT_MAX}) {
      const sgr::TileMap tm(tlo, sinks);
      const long long w = tlo / 128, s = ((long long)sinks + 127) / 128;
      const long long kept = s < w ? s : w;
      if (tm.tw != w || tm.gap != w - kept) return fail("tiles", tlo, sinks, tm.tw, tm.gap), 1;
      for (long long v = tm.gap; v < w + 3; v += v < w && kept > 4 ? kept / 4 : 1) {
        ++count;
        if (tm.at((int)v) != (v < w ? v - tm.gap : v)) return fail("tile", tlo, sinks, v, tm.at((int)v)), 1;
      }
    }
  std::printf("%lld\n", count);
  return 0;
}
