// Places of memory that overlap, against every byte of small ones.
#include <cstdio>
#include <random>
#include <set>

#include "../../parity_binade_chunked_gb300/csrc/places.h"

using namespace sq::loss;

int main() {
  std::mt19937 rng(7);
  auto any = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  int failures = 0, overlaps = 0, total = 400000;
  for (int i = 0; i < total; i++) {
    Place p[2];
    std::set<long> bytes[2];
    const int stride = any(0, 12);
    for (int k = 0; k < 2; k++) {
      const int at = any(1, 60), rows = any(0, 6), width = any(0, 9), step = any(0, 2) ? stride : any(0, 12);
      p[k] = any(0, 1) ? place((const void *)(uintptr_t)at, rows, step, width) : place((const void *)(uintptr_t)at, width);
      for (int r = 0; r < (int)p[k].rows; r++)
        for (int b = 0; b < width; b++) bytes[k].insert(at + r * (long)p[k].stride + b);
    }
    bool want = false;
    for (long b : bytes[0]) want |= bytes[1].count(b) != 0;
    overlaps += want;
    failures += overlap(p[0], p[1]) != want || overlap(p[1], p[0]) != want;
  }
  // strides and sizes whose products pass 64 bits
  const Place far = place((const void *)4096, (int64_t)1 << 27, (__int128)INT64_MAX * 4, (int64_t)1 << 26);
  failures += overlap(far, place((const void *)(uintptr_t)(4096 + (1 << 26)), 4)) || !overlap(far, place((const void *)4096, 1));
  // nothing there
  failures += overlap(place(nullptr, 100), place((const void *)1, 100)) || overlap(place((const void *)1, 0), place((const void *)1, 1));
  std::printf("failures=%d overlaps=%d of %d\n", failures, overlaps, total);
  return failures != 0;
}
