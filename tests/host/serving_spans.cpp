// Row ranges, lengths and visible keys from metadata that is not to be
// trusted, on the host: the same functions that the kernels call. Every row,
// table column and position they lead to has to lie inside its array.
#include <climits>
#include <cstdio>
#include <cstdlib>

#include "fql_serving.h"

using namespace fql;

static int64_t cases = 0;
#define CHECK(c)                                                                                             \
  do {                                                                                                       \
    if (!(c)) {                                                                                              \
      std::printf("%s: lens=%d cu=%d,%d T=%lld max_new=%d cols=%d bs=%d causal=%d window=%d\n", #c, lens[0], \
                  cu[0], cu[1], (long long)T, max_new, cols, bs, causal, window);                            \
      std::exit(1);                                                                                          \
    }                                                                                                        \
  } while (0)

static void one(int len, int c0, int c1, int64_t T, int max_new, int cols, int bs, int causal, int window) {
  const int32_t lens[1] = {len}, cu[2] = {c0, c1};
  const PagedBatch pb = {nullptr, cols, cols, lens, cu, 1, T, max_new};
  const SeqSpan s = seq_span(pb, 0, bs);
  ++cases;
  CHECK(s.row0 >= 0 && s.n >= 0 && s.n <= max_new && s.row0 + s.n <= T);
  CHECK(s.len >= 0 && s.len <= (int64_t)cols * bs && s.len <= (len < 0 ? 0 : len));
  CHECK((int64_t)s.pos0 + s.n <= INT_MAX);
  // the cache write's rows: positions from the larger of pos0 and 0 to the end
  const int64_t start = s.pos0 > 0 ? s.pos0 : 0;
  const int64_t end = (int64_t)s.pos0 + s.n < s.len ? (int64_t)s.pos0 + s.n : s.len;
  if (start < end) {
    CHECK(s.row0 + start - s.pos0 >= s.row0 && s.row0 + end - 1 - s.pos0 < s.row0 + s.n);
    CHECK((end - 1) / bs < cols);
  }
  if (s.n == 0) return;
  Visible before = {0, INT_MIN};
  for (int token : {0, s.n / 2, s.n - 1}) {
    const Visible v = visible_keys(s, token, causal, window);
    const int64_t p = (int64_t)s.pos0 + token;
    CHECK(v.hi <= s.len && v.lo >= 0);
    CHECK(!causal || v.hi <= p + 1);
    CHECK(v.lo == (window > 0 && p - window + 1 > 0 ? p - window + 1 : 0));
    CHECK(v.lo >= before.lo && v.hi >= before.hi);  // a row tile's first and last row bound the others
    before = v;
  }
}

int main() {
  const int lens[] = {INT_MIN, -1, 0, 1, 5, 15, 16, 17, 63, 64, 65, 1000, INT_MAX - 1, INT_MAX};
  const int cus[] = {INT_MIN, -7, 0, 1, 3, 16, 40, 64, 1 << 20, INT_MAX};
  const int64_t rows[] = {1, 16, 41, 1 << 20};
  for (int len : lens)
    for (int c0 : cus)
      for (int c1 : cus)
        for (int64_t T : rows)
          for (int max_new : {1, 7, 40, 1 << 20})
            for (int cols : {1, 3, 1000})
              for (int bs : {16, 64, 256})
                for (int causal : {0, 1})
                  for (int window : {0, 1, 33, 1 << 20, INT_MAX})
                    one(len, c0, c1, T, (int)(max_new < T ? max_new : T), cols, bs, causal, window);
  // the largest capacity there may be
  for (int len : lens) one(len, 0, 1 << 20, 1 << 20, 1 << 20, (1 << 30) / 256, 256, 1, 33);
  std::printf("%lld cases\n", (long long)cases);
  return 0;
}
