// Exhaustive checks of the index arithmetic of the paged attention on small
// ranges, on the CPU.  Prints "ok" and exits 0, or names the case that fails.
#include "../dual_window_attention_b200/csrc/paged_index.h"

#include <cstdio>
#include <cstdlib>
#include <vector>

using namespace ttcd;

#define REQUIRE(x)                                             \
  do {                                                         \
    if (!(x)) {                                                \
      std::printf("line %d: %s\n", __LINE__, #x);              \
      return 1;                                                \
    }                                                          \
  } while (0)

static bool sees(int t, int j, int w, int ns) { return j <= t && (j > t - w || j < ns); }

int main() {
  // key_range: every key that a position of the tile sees is in the range, every
  // key of the range before the last position's future is seen by one of them
  for (int lo = 0; lo < 14; ++lo)
    for (int hi = lo; hi < 14; ++hi)
      for (int w = 1; w < 17; ++w)
        for (int ns = 0; ns < 8; ++ns) {
          const KeyRange r = key_range(lo, hi, w, ns);
          for (int j = 0; j < 20; ++j) {
            bool any = false;
            for (int t = lo; t <= hi; ++t) any = any || sees(t, j, w, ns);
            REQUIRE(any == in_range(r, j));
          }
          for (int a = 0; a < 16; ++a)
            for (int b = a; b < 18; ++b) {
              bool any = false;
              for (int j = a; j <= b; ++j) any = any || in_range(r, j);
              REQUIRE(any == touches(r, a, b));
            }
        }
  // the largest window and position
  const KeyRange big = key_range((1 << 30) - 2, (1 << 30) - 1, 1 << 30, 128);
  REQUIRE(big.lo == 0 && big.sink_end == 0 && big.hi == (1 << 30) - 1);

  // seq_span refuses what cannot be, and never names a row or key out of range
  for (int b = -2; b < 8; ++b)
    for (int e = -2; e < 8; ++e)
      for (int L = -2; L < 8; ++L) {
        const SeqSpan s = seq_span(b, e, L, 5, 4);
        if (s.n > 0) REQUIRE(!s.bad && s.q0 >= 0 && s.q0 + s.n <= 5 && s.L <= 4 && s.L >= s.n);
        const bool fine = b >= 0 && e >= b && e <= 5 && (e == b || (L >= e - b && L <= 4));
        REQUIRE(fine == !s.bad);
        REQUIRE(!fine || s.n == e - b);
      }

  // tile slots: every tile of every sequence has a slot of its own, below the
  // bound, and the slot leads back to it
  std::srand(1);
  for (int it = 0; it < 4000; ++it) {
    const int n_seq = 1 + std::rand() % 9, tpt = 1 + std::rand() % 7;
    std::vector<int> q(1, 0);
    for (int s = 0; s < n_seq; ++s) q.push_back(q.back() + (std::rand() % 3 ? std::rand() % 13 : 0));
    const int total = q.back() + std::rand() % 5;
    const long long slots = tile_slots(total, n_seq, tpt);
    std::vector<int> seen(slots, 0);
    for (int s = 0; s < n_seq; ++s) {
      const int n = q[s + 1] - q[s];
      for (int i = 0; i * tpt < n; ++i) {
        const long long x = tile_slot(q[s], s, tpt) + i;
        REQUIRE(x >= 0 && x < slots);
        REQUIRE(seen[x]++ == 0);
        int back = -1;
        for (int u = 0; u < n_seq; ++u)
          if (tile_slot(q[u], u, tpt) <= x) back = u;
        REQUIRE(back == s);
      }
    }
  }

  // page_row: rows of distinct pages and heads do not meet and stay in the pool;
  // a page that does not exist has none
  for (int page = -3; page < 9; ++page)
    for (int h = 0; h < 3; ++h) {
      const long long r = page_row(page, 6, 3, h, 16);
      if (page < 0 || page >= 6) REQUIRE(r == -1);
      else REQUIRE(r == (page * 3 + h) * 16 && r + 15 < 6 * 3 * 16);
    }
  REQUIRE(page_row(1 << 30, 1 << 20, 8, 7, 128) == -1);
  REQUIRE(page_row((1 << 21) - 1, 1 << 21, 8, 7, 128) == ((1ll << 24) - 1) * 128);
  std::puts("ok");
  return 0;
}
