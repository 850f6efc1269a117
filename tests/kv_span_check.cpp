// Host check of kv_span (kv_layout.h) at the ends of its arguments' ranges:
// windows up to 2^63 - 1, positions from -(2^31 - 1) to 2^31 - 2. Prints "ok"
// or the first thing that is wrong.
#include <cstdio>
#include <initializer_list>

#include "kv_layout.h"

using namespace ringsim;

#define CHECK(x)                                              \
  do {                                                        \
    if (!(x)) {                                               \
      std::printf("line %d: %s\n", __LINE__, #x);             \
      return 1;                                               \
    }                                                         \
  } while (0)

int main() {
  const int64_t most = INT32_MAX;
  for (int64_t window : {most - 1, most, most + 1, (int64_t)1 << 40, INT64_MAX - 1, INT64_MAX}) {
    for (int64_t p : {-most, (int64_t)-7, (int64_t)-1, (int64_t)0, (int64_t)5, most - 2, most - 1}) {
      for (int64_t end : {(int64_t)0, (int64_t)1, (int64_t)4096, most - 1023}) {
        for (int causal = 0; causal < 2; ++causal) {
          int64_t lo, hi;
          kv_span(p, end, causal, window, &lo, &hi);
          CHECK(hi == (causal && p < end - 1 ? p : end - 1));
          // The first position that is not before the window: p - window + 1, or 0 where that would be negative.
          CHECK(lo == (p < window ? 0 : p - (window - 1)));
        }
      }
    }
  }
  std::printf("ok\n");
  return 0;
}
