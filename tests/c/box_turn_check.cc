// Host check of the epilogues' output boxes (kd_boxes.h).  A warp's transfers read
// their boxes in the order in which they were issued, as late as the waits allow:
// a box must never be staged while a transfer from it is pending.  Every sequence
// of three tiles of 1 to 8 boxes each, and long runs of equal tiles.  The rule that
// begins every tile with box 0 must be caught on the odd ones.
#include <cstdio>
#include <deque>
#include <vector>

#include "kd_boxes.h"

// Number of boxes staged while a pending transfer still reads them.
static int overwritten(const std::vector<int>& tiles, bool by_tile) {
  std::deque<uint32_t> reading;             // boxes of the transfers that have not read yet
  uint32_t turn = 0;
  int bad = 0;
  for (int boxes : tiles)
    for (int c = 0; c < boxes; ++c) {
      const uint32_t box = by_tile ? static_cast<uint32_t>(c & 1) : kd::box_take(turn);
      while (reading.size() > kd::BOX_READS_PENDING) reading.pop_front();   // the wait
      for (uint32_t r : reading) bad += r == box;
      if (box >= kd::EPI_BOXES) ++bad;
      reading.push_back(box);
    }
  return bad;
}

int main() {
  for (int a = 1; a <= 8; ++a)
    for (int b = 1; b <= 8; ++b)
      for (int c = 1; c <= 8; ++c) {
        if (overwritten({a, b, c}, false)) {
          std::printf("overwritten: tiles of %d, %d, %d boxes\n", a, b, c);
          return 1;
        }
        if ((overwritten({a, b, c}, true) != 0) != (a % 2 == 1 || b % 2 == 1)) {
          std::printf("the check does not see tiles of %d, %d, %d boxes\n", a, b, c);
          return 1;
        }
      }
  for (int n = 1; n <= 8; ++n)
    if (overwritten(std::vector<int>(10000, n), false)) return 1;
  std::printf("ok\n");
  return 0;
}
