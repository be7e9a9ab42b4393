// Drives lcb::DeviceCounts (numbers that belong to a device context, asked for
// once in each) with made-up device ordinals, context ids and answers, on the
// host. Prints "ok" and exits 0 when every check holds.
#include <cstdio>

#include "device_once.h"

static int failures = 0;
#define CHECK(cond)                                                 \
  do {                                                              \
    if (!(cond)) {                                                  \
      std::printf("check failed at line %d: %s\n", __LINE__, #cond); \
      ++failures;                                                   \
    }                                                               \
  } while (0)

int main() {
  static lcb::DeviceCounts<17> counts;
  int asked = 0;
  auto says = [&](int n) {
    return [&asked, n] {
      ++asked;
      return n;
    };
  };
  // asked once for each key of a context, and 0 is an answer
  CHECK(counts.get(0, 11, 4, says(36)) == 36 && counts.get(0, 11, 4, says(1)) == 36 && asked == 1);
  CHECK(counts.get(0, 11, 16, says(0)) == 0 && counts.get(0, 11, 16, says(1)) == 0 && asked == 2);
  // another device, and another context of the same device, have their own
  CHECK(counts.get(1, 12, 4, says(30)) == 30 && asked == 3);
  CHECK(counts.get(0, 11, 4, says(1)) == 36 && asked == 3);
  CHECK(counts.get(0, 13, 4, says(20)) == 20 && counts.get(0, 13, 4, says(1)) == 20 && asked == 4);
  // a query that failed counts as 0 and is asked again
  CHECK(counts.get(2, 14, 8, says(-1)) == 0 && asked == 5);
  CHECK(counts.get(2, 14, 8, says(15)) == 15 && asked == 6);
  CHECK(counts.get(2, 14, 8, says(-1)) == 15 && asked == 6);
  // no context id, ids and ordinals outside the table, counts too large for it: asked every time
  CHECK(counts.get(3, 0, 2, says(5)) == 5 && counts.get(3, 0, 2, says(6)) == 6 && asked == 8);
  CHECK(counts.get(-1, 9, 2, says(5)) == 5 && counts.get(lcb::kMaxDeviceOrdinals, 9, 2, says(6)) == 6 && asked == 10);
  CHECK(counts.get(3, 1ull << 48, 2, says(5)) == 5 && counts.get(3, 1ull << 48, 2, says(6)) == 6 && asked == 12);
  CHECK(counts.get(3, 15, 2, says(1 << 16)) == 1 << 16 && counts.get(3, 15, 2, says(7)) == 7 && asked == 14);
  if (failures) return 1;
  std::printf("ok\n");
  return 0;
}
