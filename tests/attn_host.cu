// Host check of the attention kernels' index arithmetic (run by
// tests/test_attn_cpu.py): which tiles a sequence's rows read, what the
// device's checks of its tables let through, and how runs cut the unit list.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>

#include <algorithm>

#include "../include/moe.h"
#include "attn_prefill.cuh"

using namespace moe;

#define CHECK(x)                                              \
  do {                                                        \
    if (!(x)) {                                               \
      std::printf("line %d: %s\n", __LINE__, #x);             \
      std::exit(1);                                           \
    }                                                         \
  } while (0)

static void tiles() {
  const int kvs[] = {1, 2, 63, 64, 65, 127, 128, 129, 200, 640, 1000};
  const int windows[] = {0, 1, 2, 63, 64, 65, 100, 999, 1000, 5000, 2147483647};
  const int sinks[] = {0, 1, 4, 63, 64, 65, 130, 2147483647};
  for (int kv : kvs)
    for (int rows : {1, 2, 5, 32, 64, 65, 1000})
      for (int w : windows)
        for (int sk : sinks) {
          if (rows > kv) continue;
          const SeqView s = seq_check(0, rows, kv, rows, (kv + 15) / 16, 16);
          CHECK(s.ok && s.rows == rows && s.kv == kv);
          const SeqTiles t = seq_tiles(s, w, sk);
          std::set<int> got;
          int before = -1;
          for (int k = 0; k < t.n; ++k) {
            const int tile = tile_at(t, k);
            CHECK(tile > before && tile >= 0 && tile * kAtTile < kv);
            before = tile;
            got.insert(tile);
          }
          std::set<int> again;
          for (int k = 0; k < t.n; ++k) again.insert(tile_at_lead_last(t, k));
          CHECK(again == got);
          std::set<int> want;
          for (int j = 0; j < kv; ++j) {
            bool seen = false;
            for (int i = kv - rows; i < kv && !seen; ++i)
              seen = j <= i && (w <= 0 || i - j < w || j < sk);
            if (seen) want.insert(j / kAtTile);
          }
          for (int j = 0; j < kv + 70; j += 16) {  // a page is needed when one of its keys is seen
            bool seen = false;
            for (int x = j; x < j + 16 && x < kv && !seen; ++x)
              for (int i = kv - rows; i < kv && !seen; ++i) seen = x <= i && (w <= 0 || i - x < w || x < sk);
            CHECK(seen == keys_seen(s, w, sk, j, 16));
          }
          for (int x : want) CHECK(got.count(x));
          CHECK(got.size() <= want.size() + 1);
        }
}

static void tables() {
  const int odd[] = {-2147483647 - 1, -5, -1, 0, 1, 3, 4, 5, 64, 65, 2147483647};
  const int n_rows = 4, max_pages = 4, page = 16;
  for (int a : odd)
    for (int b : odd)
      for (int kv : odd) {
        const SeqView s = seq_check(a, b, kv, n_rows, max_pages, page);
        if (!s.ok) {
          CHECK(s.rows == 0 && s.kv == 0);
          CHECK(seq_tiles(s, 0, 0).n == 0);
          continue;
        }
        CHECK(s.row0 >= 0 && s.row0 + s.rows <= n_rows && s.rows >= 0);
        CHECK(s.kv >= s.rows && s.kv <= max_pages * page);
      }
}

// Every unit belongs to one block; a segment's parts are the blocks first ..
// last, each with a slot of its own.
static void runs() {
  for (int grid : {1, 2, 7, 296})
    for (int min_units : {1, 2, 4})
      for (int trial = 0; trial < 60; ++trial) {
        std::vector<long long> seg;
        long long total = 0;
        for (int i = 0; i <= trial; ++i) {
          seg.push_back(1 + (i * 7919 + trial * 104729) % (1 + trial * 9));
          total += seg.back();
        }
        const long long run = run_length(total, grid, min_units);
        CHECK(run * grid >= total && run >= min_units);
        std::set<long long> slots;
        std::set<int> keys;
        long long u = 0;
        for (long long n : seg) {
          const int first = (int)(u / run), last = (int)((u + n - 1) / run);
          CHECK(last < grid);
          if (first != last) {
            CHECK(keys.insert(first).second);  // one arrival counter per split segment
            for (int b = first; b <= last; ++b) CHECK(slots.insert(b * 2LL + (b == first)).second);
          }
          u += n;
        }
      }
}

// The parts of a block's tiles: none empty, together all, no more than asked.
static void key_ranges() {
  for (int n = 1; n < 3000; n = n < 300 ? n + 1 : n * 2)
    for (int most : {1, 2, 3, 7, 37, 148}) {
      const int k = key_parts(n, most);
      CHECK(k >= 1 && k <= most);
      int at = 0;
      for (int i = 0; i < k; ++i) {
        const int lo = (int)((long long)n * i / k), hi = (int)((long long)n * (i + 1) / k);
        CHECK(lo == at && hi > lo);
        at = hi;
      }
      CHECK(at == n);
    }
}

int main() {
  key_ranges();
  tiles();
  tables();
  runs();
  std::puts("ok");
  return 0;
}
