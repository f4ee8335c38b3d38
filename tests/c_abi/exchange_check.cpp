// The marks of exchange.h: none is another launch's, none can stand in finite data, and a word gives its value back.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <vector>
#include <algorithm>

#include "exchange.h"

using namespace qlora;

int main() {
  int bad = 0;
  std::vector<uint64_t> marks;
  const uint64_t starts[] = {0, 1000, 0xffffff00u, (uint64_t)5 << 32, ((uint64_t)1 << 39) - 1000};
  for (uint64_t s : starts)
    for (uint64_t i = 0; i < 1000; ++i) marks.push_back(exchange_mark(s + i));
  std::vector<uint64_t> sorted = marks;
  std::sort(sorted.begin(), sorted.end());
  // 0xffffff00 + i overlaps nothing of the others
  for (size_t i = 1; i < sorted.size(); ++i) bad += exchange_holds(sorted[i - 1], sorted[i]);
  std::printf("shared marks %d\n", bad);
  int finite = 0, lost = 0;
  for (uint64_t m : marks)
    for (uint32_t v : {0u, 1u, 0x7fffu, 0x8000u, 0xffffu}) {
      const uint64_t w = exchange_word(m, v | 0xabcd0000u);
      lost += !exchange_holds(w, m) || (uint32_t)(w & 0xffff) != v;
      const uint32_t low = (uint32_t)w, bf16 = (uint32_t)w & 0xffff0000u;
      float f, h;
      std::memcpy(&f, &low, 4);
      std::memcpy(&h, &bf16, 4);
      finite += std::isfinite(f) || std::isfinite(h);
    }
  std::printf("finite %d lost %d zero %d\n", finite, lost, (int)exchange_holds(0, marks[0]));
  return bad || finite || lost;
}
