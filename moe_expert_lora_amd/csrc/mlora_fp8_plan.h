// In which tiles a call of the 8-bit products is cut. Plain host code of sizes alone.
#ifndef MLORA_FP8_PLAN_H_
#define MLORA_FP8_PLAN_H_

#include <algorithm>
#include <cstdint>

namespace mlora {

// Waves of 16 x 16 that read their operands straight from memory, or tiles through LDS.
enum Fp8Form { kFp8Stream, kFp8Rows32, kFp8Rows64, kFp8Rows128, kFp8Rows256 };

// The form goes by the rows that a span has on average and by the tiles that they make:
// larger tiles reuse more, but a span's last tile is half empty and the chip's 256 CUs
// want two workgroups each (one of 256 x 256, which fills a CU's LDS). Every form was
// measured on 265 calls: one weight of 2048 x 40 to 1000 x 6000 with 20 to 20000 rows, and
// spans of 5 to 800 rows of 4 to 384 experts, routed evenly and skewed. The rule is 1.1%
// from the fastest form on average with fp32 sums, 1.4% with fast ones, 24% at most. Its
// edges lie where the forms cross, flat over the ranges in brackets; us on both sides:
//   stream -> 32 rows: 1536 tiles of 16 x 16, six a CU (1400 to 1700)
//     1440: 21.1, 23.0   1536: 9.1, 9.4   2016: 22.9, 18.3   2080: 37.8, 23.7
//   32 -> 64, fp32 sums: 32 rows a span (28 to 36), 320 tiles of 64 x 128 (300 to 384)
//     24 rows, skewed: 15.3, 18.0   36: 39.2, 32.6   288 tiles: 15.4, 17.1   384: 44.2, 39.0
//   32 -> 64, fast: 24 rows (24 to 32), 256 tiles (200 to 290)
//     20 rows: 38.2, 40.4   36: 46.6, 42.9   192 tiles: 17.1, 17.6   312: 25.0, 18.4
//   64 -> 128, fp32 sums: 200 rows (160 to 200), 512 tiles of 128 x 128 (500 to 770)
//     180 rows: 92.8, 102.7   200: 123.4, 115.3   384 tiles: 55.1, 62.0   752: 34.0, 30.4
//   64 -> 128, fast: 64 rows (50 to 70), 320 tiles (290 to 330)
//     50 rows: 106.9, 122.1   70: 54.8, 49.8   192 tiles: 24.3, 28.7   480: 64.6, 45.4
//   128 -> 256, fast alone: 128 rows (100 to 130), 192 tiles of 256 x 256 (140 to 200)
//     90 rows: 144.4, 153.6   130: 71.9, 57.1   128 tiles: 14.7, 19.0   256: 33.6, 27.2
// fp32 sums take twice the matrix instructions, and the largest tile has nothing left to
// save there (8192 rows of one 4096 x 4096: 244 of 128 x 128, 261 of 256 x 256 with
// registers spilled): they do not have it.
inline Fp8Form plan_fp8(int64_t n_rows, int64_t n_experts, int64_t n_out, bool fast) {
  const int64_t spans = std::min(n_experts, n_rows), mean = (n_rows + spans - 1) / spans;
  auto tiles = [&](int64_t bm, int64_t bn) {
    return spans * ((mean + bm - 1) / bm) * ((n_out + bn - 1) / bn);
  };
  if (2 * tiles(16, 32) < 1536) return kFp8Stream;
  if (fast && mean >= 128 && tiles(256, 256) >= 192) return kFp8Rows256;
  if (mean >= (fast ? 64 : 200) && tiles(128, 128) >= (fast ? 320 : 512)) return kFp8Rows128;
  if (mean >= (fast ? 24 : 32) && tiles(64, 128) >= (fast ? 256 : 320)) return kFp8Rows64;
  return kFp8Rows32;
}

}  // namespace mlora

#endif  // MLORA_FP8_PLAN_H_
