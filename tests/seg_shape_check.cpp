// Which output tile a product by expert or with 4-bit operands gets.  First
// what has to hold for every size, over many of them; then, for each line of
// the input, the tile:
//   rows M N experts segments fp4 words      depth M N experts
// Prints the first mistake and fails.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include "seg_shape.h"

using namespace fp8sg;

// a launch's workgroups, less the rest of a round over 8; the workspace's words
static const int64_t kGrid = (1 << 22) - 7, kWords = 1 << 16;

static void need(bool ok, const char* what, const SegSize& q) {
  if (ok) return;
  std::printf("%s: %lld x %lld, %d experts, segments %d, 4 bits %d\n", what, (long long)q.M,
              (long long)q.N, q.experts, q.segments, q.fp4);
  std::exit(1);
}

// Tile rows of M rows in `used` segments, all but one of them one row more
// than a multiple of bm where there are rows enough.
static int64_t worst(int64_t M, int used, int bm) {
  if (used == 0) return 0;
  int64_t left = M - used, tiles = 0;
  for (int i = 0; i + 1 < used; ++i) {
    const int64_t more = left >= bm ? bm : 0;
    left -= more;
    tiles += (1 + more + bm - 1) / bm;
  }
  return tiles + (1 + left + bm - 1) / bm;
}

static void walk() {
  const int64_t Ms[] = {1, 2, 16, 17, 24, 25, 32, 33, 64, 65, 176, 177, 320, 321, 1000, 4096, 24576,
                        24577, 65536, 262144, 2147483647};
  const int64_t Ns[] = {1, 16, 64, 65, 128, 1929, 2313, 11008, 49152, 174784, 262400, 4194304, 4194320};
  const int Es[] = {1, 2, 8, 63, 64, 65, 128, 1024};
  for (int64_t M : Ms)
    for (int64_t N : Ns)
      for (int e : Es)
        for (int f = 0; f < 4; ++f) {
          const SegSize q{M, N, f & 1 ? e : 1, (f & 1) != 0, (f & 2) != 0};
          for (int64_t words : {(int64_t)0, kWords}) {
            const TileKind t = choose_rows(q, kGrid, words);
            need(t >= kTile16 && t <= kTile256, "no such tile", q);
            need(t != kTile16 || q.fp4, "16 rows are for 4 bits", q);
            need(t == kTile256 || row_tiles(q, t) <= kGrid, "more tiles than a grid", q);
            need(!words || t == kTile256 || row_tiles(q, t) <= words, "more maxima than words", q);
            if (!q.segments || M > 1 << 20) continue;
            const int bm = size_of(t).rows;
            const int64_t columns = (N + size_of(t).columns - 1) / size_of(t).columns;
            for (int used = 0; used <= q.experts && used <= M; used = used * 2 + 1)
              need(worst(M, used, bm) * columns <= row_tiles(q, t), "tiles without a workgroup", q);
          }
        }
}

int main() {
  static const char* const names[] = {"16x64", "32x64", "64x64", "64x128", "128x128", "256x256"};
  for (int t = kTile16; t <= kTile256; ++t) {
    char name[16];
    std::snprintf(name, sizeof name, "%dx%d", size_of((TileKind)t).rows, size_of((TileKind)t).columns);
    if (std::strcmp(name, names[t]) != 0) return std::printf("size of %s\n", names[t]), 1;
  }
  walk();
  char kind[8];
  while (std::scanf("%7s", kind) == 1) {
    long long M, N, words = 0;
    int experts, segments = 1, fp4 = 0;
    const bool rows = std::strcmp(kind, "rows") == 0;
    if (std::scanf("%lld %lld %d", &M, &N, &experts) != 3) return 1;
    if (rows && std::scanf("%d %d %lld", &segments, &fp4, &words) != 3) return 1;
    const SegSize q{M, N, experts, segments != 0, fp4 != 0};
    std::puts(names[rows ? choose_rows(q, kGrid, words) : choose_depth(q)]);
  }
  return 0;
}
