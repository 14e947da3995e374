// Checks of the unit slots of the paged attention's kernel of few rows, on the
// CPU.  Prints "ok" and exits 0, or names the case that fails.
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

int main() {
  // every unit after a sequence's first has an extra slot of its own, below the
  // bound, and the slot leads back to it
  std::srand(2);
  for (int it = 0; it < 20000; ++it) {
    const int n_seq = 1 + std::rand() % 9, tpt = 1 + std::rand() % 8;
    std::vector<int> q(1, 0);
    for (int s = 0; s < n_seq; ++s) q.push_back(q.back() + (std::rand() % 3 ? std::rand() % 20 : 0));
    const int total = q.back() + std::rand() % 5;
    std::vector<int> seen(extra_slot(total, tpt), 0);
    for (int x = 0; x < extra_slot(total, tpt); ++x) {
      int s = -1;
      for (int u = 0; u < n_seq; ++u)
        if (extra_slot(q[u], tpt) <= x) s = u;
      REQUIRE(s >= 0);
      const int tok = extra_token(x, q[s], tpt);
      REQUIRE(tok >= tpt && tok % tpt == 0);
      if (tok < q[s + 1] - q[s]) seen[x] = s * 1000 + tok;
    }
    for (int s = 0; s < n_seq; ++s)
      for (int tok = tpt; tok < q[s + 1] - q[s]; tok += tpt) {
        const int x = extra_slot(q[s], tpt) + tok / tpt - 1;
        REQUIRE(x < extra_slot(total, tpt) && seen[x] == s * 1000 + tok);
      }
  }
  // starts that cannot be do not wrap round
  REQUIRE(extra_token((1 << 30) - 1, -2147483647 - 1, 8) == 1 << 30);
  std::puts("ok");
  return 0;
}
