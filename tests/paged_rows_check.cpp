// Checks on the CPU that a row of the packed queries leads to a token of its sequence
// or to none, for starts and lengths up to the ends of 32 bits.  Prints "ok" and exits 0,
// or names the case that fails.
#include "../dual_window_attention_b200/csrc/paged_index.h"

#include <climits>
#include <cstdio>

using namespace ttcd;

int main() {
  const int ends[] = {INT_MIN, INT_MIN + 1, -(1 << 30), -1, 0, 1, 2, 5, 6, 1 << 30, INT_MAX - 1, INT_MAX};
  const int total = 6;
  const long long capacity = 32;
  for (int begin : ends)
    for (int end : ends)
      for (int kv_len : ends)
        for (int row = 0; row < total; ++row) {
          const SeqSpan s = seq_span(begin, end, kv_len, total, capacity);
          const int tok = row_token(s, row);
          const bool holds = !s.bad && begin <= row && row < end;
          if (holds ? tok != row - begin : tok != -1) {
            std::printf("row %d of [%d, %d) with %d keys: token %d\n", row, begin, end, kv_len, tok);
            return 1;
          }
          if (tok >= 0) {  // its position has a page in the table
            const int p = s.L - s.n + tok;
            if (p < 0 || p >= capacity) {
              std::printf("row %d of [%d, %d) with %d keys: position %d\n", row, begin, end, kv_len, p);
              return 1;
            }
          }
        }
  std::puts("ok");
  return 0;
}
