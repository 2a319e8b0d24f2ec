// How a call of the 4-bit products is laid over workgroups and waves: which of
// the two forms of mlora_w4.hip, and in which shape. Plain host code of sizes
// alone.
#ifndef MLORA_W4_PLAN_H_
#define MLORA_W4_PLAN_H_

#include <cstdint>

#include "mlora.h"

namespace mlora {

constexpr int kScan = 2048;                // rows scanned (and listed) at a time
constexpr int kSplitWaves = 8;             // most per workgroup, split form
constexpr int kMaxWaves = 12;              // of both

// Streaming form.
constexpr int kPair = 2;   // tiles per wave and step
// Chunks in flight per wave: a CU's cache has lines for 32 KB of loads on their
// way, which 12 waves' chunks of two tiles fill; further ones wait at the cache,
// and hold registers (3 instead of 2: 128 experts of 2048 x 768, 2048 rows 30.2 ->
// 30.9 us, with groups of 32 34.5 -> 35.7; 4: 31.1 and 43.7).
constexpr int kAhead = 2;
constexpr int kLds = 160 * 1024;        // of a CU
constexpr int kListLds = kScan * 4 + 256;  // the list and the counts
// A chunk of x rows: the operands and the groups' sums.
constexpr int chunk_lds(bool f32, int mb, int sg) {
  return mb * (4 * (f32 ? 3 : 1) * 1024 + sg * 64);
}
// Chunks of x rows that fit a workgroup's LDS.
constexpr int panel_chunks(bool f32, int mb, int sg) {
  return (kLds - kListLds) / chunk_lds(f32, mb, sg);
}

// Waves a SIMD holds: what the registers are kept to.
constexpr int simd_waves(bool f32, int mb) { return f32 || mb > 1 ? 3 : 4; }

// The rows of a call. They lead a kernel's arguments as plain values, which
// arrive in registers, so that the scan does not wait for the others.
struct W4Rows {
  const int32_t* ids;  // null: one weight
  int32_t n, experts;
};

struct W4Plan {
  bool stream, by_row;
  int places, mb, tiles, waves, k_waves, splits, per_slice, slices;
};

inline W4Plan plan_w4(const mlora_w4_route* r, W4Rows rows, bool f32, int sg) {
  W4Plan p{};
  p.k_waves = 1;
  const int64_t tiles = (r->n_out + 15) / 16, chunks = (r->k_in + 127) / 128;
  p.by_row = rows.ids && rows.n < rows.experts;
  const int64_t places = p.by_row ? rows.n : rows.experts;
  p.places = (int)places;
  const int64_t mean = (rows.n + places - 1) / places;  // rows per place
  // Row blocks of 16 per pass over the weights: two once an expert holds more
  // than ten rows on average.
  p.mb = !f32 && (places == 1 ? mean > 16 : mean > 10) ? 2 : 1;
  const int64_t blocks = (mean + 16 * p.mb - 1) / (16 * p.mb);  // passes
  const int64_t pairs = (tiles + kPair - 1) / kPair;
  // Streaming pays from 512 pairs of tiles (16 experts of 1024 x 1024, 64 rows, 512
  // pairs: 9.2 us, split 10.2; 60 of 512 x 200, 420 pairs: 8.2, split 6.0), or from
  // fewer of long k (4 of 4000 x 4000, 500 pairs of 32 chunks, 64 rows: 19.8, split
  // 26.3; 60 of 2048 x 200, 420 of 16 chunks: 10.5, split 10.4).
  p.stream = places * pairs >= 512 || places * pairs * chunks >= 8192;
  if (p.stream) {
    const int64_t most = panel_chunks(f32, p.mb, sg);
    const int64_t x_lds = (chunks < most ? chunks : most) * chunk_lds(f32, p.mb, sg);
    // Two workgroups a CU, where x leaves room for them, cover each other's starts
    // (128 experts of 768 x 2048, 640 rows: 21.5 us in eights, 22.6 in twelves); one
    // alone has twelve waves (20 of 4000 x 4000, 60 rows: 34.5 us, in eights 40).
    const int64_t per_simd = simd_waves(f32, p.mb);
    const int64_t most_waves = per_simd == 4 && 2 * (x_lds + kListLds) <= kLds ? 8 : kMaxWaves;
    auto room = [&](int64_t waves, int kw) {  // workgroups the CUs hold at once
      int64_t lds = x_lds;
      const int64_t sums = waves * kPair * p.mb * 1024;
      if (kw > 1 && lds < sums) lds = sums;
      const int64_t by_lds = kLds / (lds + kListLds), by_reg = per_simd / ((waves + 3) / 4);
      return 256 * (by_lds < by_reg ? by_lds : by_reg);
    };
    // All pairs at once, as many waves to a pair as k has chunks for, until a CU has
    // eight: their requests fill its cache's lines (64 experts of 4096 x 512, 128
    // rows, 1024 pairs: 1, 2, 3 waves to a pair 19.8, 16.4, 17.7 us; 4 of 4000 x
    // 4000, 8 rows, 500 pairs: 20.1, 14.5, 13.6, with four 12.3) ...
    for (int kw = 4; kw >= 1 && p.waves == 0; --kw) {
      if (kw > 1 && (chunks < 3 * kw || kAhead * kw > most)) continue;
      if (kw > 1 && places * pairs * (kw - 1) >= 256 * 8) continue;
      for (int64_t wn = 1; wn * kw <= most_waves; ++wn) {
        if (wn * kw < 4) continue;
        const int64_t slices = (pairs + wn - 1) / wn;
        if (places * slices > room(wn * kw, kw)) continue;
        p.k_waves = kw;
        p.waves = (int)(wn * kw);
        p.slices = (int)slices;
        p.per_slice = (int)wn;
        break;
      }
    }
    // ... or several pairs per wave one after the other, in one round of
    // workgroups (one pair where k takes several panels, whose sums stay in
    // registers)
    if (p.waves == 0) {
      p.waves = (int)most_waves;
      int64_t slices = room(p.waves, 1) / places;
      if (slices < 1) slices = 1;
      if (chunks > most || slices > (pairs + p.waves - 1) / p.waves)
        slices = (pairs + p.waves - 1) / p.waves;
      p.per_slice = (int)((pairs + slices - 1) / slices);
      p.slices = (int)((pairs + p.per_slice - 1) / p.per_slice);
    }
  } else {
    const int64_t per = (chunks + kSplitWaves - 1) / kSplitWaves;
    p.waves = (int)((chunks + per - 1) / per);
    // Two tiles a workgroup where several passes over the rows fill the CUs: x,
    // which each workgroup reads whole, is then what moves (one weight of 4000 x
    // 4000, 44 rows: 14.0 us with one tile, 11.2 with two; 24 rows, one pass: 8.7
    // and 10.2; 2048 x 2048, 44 rows: 6.9 and 7.4).
    p.tiles = blocks >= 2 && places * tiles * blocks > 320 ? 2 : 1;
    p.slices = (int)((tiles + p.tiles - 1) / p.tiles);
  }
  // Rows of one expert over several workgroups: once an expert holds more than
  // two passes on average, or while there are less than two workgroups a CU (one
  // weight of 4000 x 4000, 24 rows of fp32: 17.7 us in one workgroup per tile,
  // 13.4 in two). More, for the experts above the average, gave nothing.
  const int64_t wgs = places * p.slices;
  int64_t splits = blocks <= 2 ? 1 : (blocks + 1) / 2;
  if (splits < blocks && wgs * splits < 512) splits = blocks < 512 / wgs + 1 ? blocks : 512 / wgs + 1;
  p.splits = (int)(splits > 32 ? 32 : splits);
  return p;
}

}  // namespace mlora

#endif  // MLORA_W4_PLAN_H_
