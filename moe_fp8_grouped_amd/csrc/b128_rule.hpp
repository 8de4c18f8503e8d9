// Which kernel a grouped product in blocks of 128 runs: a rule on sizes alone,
// plain C++ so that a host test can ask it too.
#pragma once

#include <stdint.h>

namespace moe {
namespace b128 {

// Results of a wide tile (gmm: uneven groups of 256 rows on average mostly fit one tile of 320; 288 rows took the slice
// 294 us where 320 took 291), and of a narrow one.
constexpr int kWideRowsGmm = 320, kWideRowsTgmm = 256, kWideCols = 256, kNarrow = 64;

enum Choice { kFew16, kFew32, kFew64, kNarrowTiles, kWideTiles };

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles of the few-rows kernel with `rows` rows each: one more than any split of M rows into the groups makes.
inline int64_t few_tiles(int64_t El, int64_t M, int rows) {
  return El == 1 ? ceil_div(M, rows) : M / rows + (El < M ? El : M) + 1;
}

// The few-rows kernel as long as its 16 x 16 pieces are at most six a CU.  One group of 7168 by 4096: 1 row 8.2 us (narrow
// tiles 27), 64 rows 23 (33), 128 rows 42 (33); 64 groups of 2048 by 1536: 8 rows 11 (12), 16 rows 19 (19), 32 rows 31 (26).
//
// Wide tiles where every workgroup has one: 128 rows in 64 groups of 2048 x 1536 take 41 us (narrow ones 44 to 47), the weight
// gradient of 512 rows in 8 groups, 2080 x 1040, 19 us (narrow ones 29); 512 rows in 8 groups of 2080 x 1040, 20 tiles, take 12.4 us
// with narrow ones (wide ones 22), 2048 rows in 8 groups of 2048 x 1536, 84 tiles, 30 (35).  The rule errs where tiles are full and
// somewhat fewer than CUs (one group of 4096 rows, 8192 x 4096, 208 tiles: 493 us, wide ones 136; of 2048 rows, 4096 x 4096, 112
// tiles: 131, wide ones 71; of 1024, 64 tiles: 67 and 61), and where rows, which it cannot see, are in few of the groups that it
// counts (128 rows in one of 64 groups of 2048 x 1536: 25 us, narrow ones 12; 2048 in one: 39 and 29; evenly: 38 and 43).
inline Choice product_kernel(int64_t El, int64_t M, int64_t N, int cus) {
  const int rows = El == 1 && M > 32 ? 64 : El == 1 && M > 16 ? 32 : 16;
  if (few_tiles(El, M, rows) * (N / 16) * (rows / 16) <= 6 * static_cast<int64_t>(cus)) return rows == 64 ? kFew64 : rows == 32 ? kFew32 : kFew16;
  return ((El < M ? El : M) + M / kWideRowsGmm) * ceil_div(N, kWideCols) >= cus ? kWideTiles : kNarrowTiles;
}
inline Choice gradient_kernel(int64_t El, int64_t K, int64_t N, int cus) {
  return El * ceil_div(K, kWideRowsTgmm) * ceil_div(N, kWideCols) >= cus ? kWideTiles : kNarrowTiles;
}

}  // namespace b128
}  // namespace moe
