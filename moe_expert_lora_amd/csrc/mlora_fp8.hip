// Products with 8-bit floating-point expert weights (OCP E4M3, a scale for each
// block of 128 x 128), for gfx950 (MI355X): the weights' layout, the rows'
// quantiser, and the product over rows sorted by expert.
#include "mlora_fp8.h"
#include "mlora_fp8_plan.h"
#include <type_traits>

namespace mlora {
namespace {

// ---------------------------------------------------------------------------
// pack
// ---------------------------------------------------------------------------
//
// A thread moves the 16 bytes of one lane and half (mlora_fp8.h). Forward, they
// lie together in the source row, at any address. Transposed, a workgroup takes its
// block of 128 x 128 through LDS: rows of 128 neighbouring columns in, each thread's 16
// bytes of a column out.
// 128 weights of 2048 x 768 (201 MB each way): 77 to 96 us, transposed 76 (5.2 TB/s).

struct Fp8PackArgs {
  const uint8_t* w;
  const float* scales;
  uint8_t* packed;
  float* packed_scales;
  int64_t cells;          // blocks, of as many scales
  int32_t N, K, NB, KB;   // of the packed (transposed) matrix
  int32_t transpose;
};

typedef u32x4 u32x4_byte __attribute__((aligned(1)));

// 16 bytes of a row of `len` from `at` on, zeros past it.
__device__ __forceinline__ u32x4 load_codes(const uint8_t* row, int at, int len) {
  u32x4 v = {0, 0, 0, 0};
  if (at >= len) return v;
  if (at + 16 <= len) return *reinterpret_cast<const u32x4_byte*>(row + at);
#pragma unroll
  for (int j = 0; j < 15; ++j)
    if (at + j < len) v[j / 4] |= (uint32_t)row[at + j] << (8 * (j % 4));
  return v;
}

// Chunk c of a block of 128 x 128, 1024 of them: its column and its first k.
__device__ __forceinline__ void pack_place(int c, int nb, int kb, int* n, int* k) {
  const int lane = c & 63, half = (c >> 6) & 1, part = c >> 7, r = lane & 15;
  *n = fp8_column(nb * 8 + part, r >> 2) + (r & 3);
  *k = kb * 128 + (lane >> 4) * 32 + half * 16;
}

// One workgroup a block and its scale.
__global__ void __launch_bounds__(256) fp8_pack_kernel(Fp8PackArgs a) {
  __shared__ uint8_t tile[128][132];  // [k][n], transposed weights
  const int64_t block = flat_group();
  if (block >= a.cells) return;
  const int tid = threadIdx.x;
  const int kb = (int)(block % a.KB);
  const int64_t t = block / a.KB;
  const int nb = (int)(t % a.NB);
  const int64_t e = t / a.NB;
  const uint8_t* w = a.w + e * a.N * a.K;
  if (tid == 0)
    a.packed_scales[block] = a.scales[e * a.NB * a.KB + (a.transpose ? (int64_t)kb * a.NB + nb
                                                                     : (int64_t)nb * a.KB + kb)];
  uint8_t* out = a.packed + block * (8 * kFp8Tile);
  if (a.transpose) {
    const int n = tid % 8 * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = i * 32 + tid / 8;
      u32x4 v = {0, 0, 0, 0};
      if (kb * 128 + k < a.K)
        v = load_codes(w + (int64_t)(kb * 128 + k) * a.N, nb * 128 + n, a.N);
#pragma unroll
      for (int j = 0; j < 4; ++j) *reinterpret_cast<uint32_t*>(&tile[k][n + 4 * j]) = v[j];
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = i * 256 + tid;
    int n, k;
    pack_place(c, nb, kb, &n, &k);
    u32x4 v = {0, 0, 0, 0};
    if (a.transpose) {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j / 4] |= (uint32_t)tile[k % 128 + j][n % 128] << (8 * (j % 4));
    } else if (n < a.N) {
      v = load_codes(w + (int64_t)n * a.K, k, a.K);
    }
    *reinterpret_cast<u32x4*>(out + c * 16) = v;
  }
}

// ---------------------------------------------------------------------------
// quantise rows
// ---------------------------------------------------------------------------
//
// A group of 128 values of a row: m = its largest magnitude (448 * 2^-126 at
// least), scale = m / 448, code = 448 x / m to the nearest E4M3 value, ties to
// even. 16 lanes hold a group, 8 values each. silu(x) up is an fp32 value, each of its
// operations rounded. The codes are those of the exact quotient:
// - x in bf16: with e the exponent of m, both 448 x 2^-e (exact) and m 2^-e in [1, 2)
//   are fp32 values, and a quotient by the rounded reciprocal, corrected once by its
//   remainder, is the correctly rounded one; x and m have 8 bits each, so a quotient
//   that is not half way between two codes stays off that border by more than fp32's
//   rounding.
// - fp32 values: a product with 448 / m is within 2 units of the exact quotient. Where
//   2^-20 less and 2^-20 more of it give the same codes, they are the exact one's; a lane
//   of others (one in 10000) divides in fp64 and keeps what the rounding to fp32 cuts off
//   in the last bit. 32768 rows of 768 with silu take 32 to 36 us (47 where every lane
//   divides in fp64; 30 of silu by a reciprocal), 8192 fp32 rows of 2048 14.8 (16.6).
// A group with an infinity or NaN gets a NaN as scale and codes of 0.

struct QuantArgs {
  const void* x;
  int64_t x_ld;
  const void* up;  // null: x itself
  int64_t up_ld;
  uint8_t* q;
  int64_t q_ld;
  float* scales;   // [groups][n_rows]
  uint32_t units;  // n_rows * groups
  int32_t n_rows, K, groups;
};

// Four E4M3 codes, the first in the low byte.
__device__ __forceinline__ uint32_t pack_fp8(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return (uint32_t)v;
}

template <typename Row, bool SILU>
__global__ void __launch_bounds__(256) fp8_quant_kernel(QuantArgs a) {
  const uint32_t unit = (uint32_t)flat_group() * 16 + (threadIdx.x >> 4);
  if (unit >= a.units) return;  // whole rows of 16 lanes: the reduction stays in them
  const int row = (int)(unit / (uint32_t)a.groups);
  const int g = (int)(unit - (uint32_t)row * (uint32_t)a.groups);
  typedef typename Row::elem elem;
  const int k[1] = {g * 128 + (int)(threadIdx.x & 15) * 8};
  Eights<Row, 1> x, up;
  x.request(static_cast<const elem*>(a.x) + (int64_t)row * a.x_ld, k, a.K);
  if constexpr (SILU) up.request(static_cast<const elem*>(a.up) + (int64_t)row * a.up_ld, k, a.K);
  float v[8];
  x.finish(k, a.K);
  x.widen(0, v);
  if constexpr (SILU) {
    float u[8];
    up.finish(k, a.K);
    up.widen(0, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = silu(v[i]) * u[i];
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  m = group_max<16>(m);
  const bool bad = m >= 0x7f800000u;
  m = bad ? 0x3f800000u : max(m, 0x04e00000u);  // 448 * 2^-126 = 1.75 * 2^-118
  const float top = __uint_as_float(m);
  const int e = (int)(m >> 23) - 127;
  const float den = __uint_as_float((m & 0x7fffffu) | 0x3f800000u);
  const float num = ldexpf(448.f, -e);
  const float r = 1.f / den;
  float c[8];
  auto pack = [&] {
    return u32x2{pack_fp8(c[0], c[1], c[2], c[3]), pack_fp8(c[4], c[5], c[6], c[7])};
  };
  u32x2 out;
  if constexpr (sizeof(typename Row::elem) == 2 && !SILU) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = v[i] * num;
      const float q = t * r;
      c[i] = fmaf(fmaf(-q, den, t), r, q);
    }
    out = pack();
  } else {
    const float scale = num * r;
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = v[i] * scale * (1.f - 0x1p-20f);
    const u32x2 low = pack();
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = v[i] * scale * (1.f + 0x1p-20f);
    out = pack();
    if (low[0] != out[0] || low[1] != out[1]) {
      const double rd = 1.0 / (double)top;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double t = (double)v[i] * 448.0 * rd;
        const float f = (float)t;
        // an even last bit with something cut off: one step towards it
        const double off = t - (double)f;
        const uint32_t b = __float_as_uint(f);
        const bool odd = (b & 1u) || fabs(off) <= fabs(t) * 0x1p-40;
        const bool grow = (off > 0.0) == (f > 0.f);
        c[i] = odd || f == 0.f ? f : __uint_as_float(grow ? b + 1u : b - 1u);
      }
      out = pack();
    }
  }
  if (bad) out = u32x2{0, 0};
  *reinterpret_cast<u32x2*>(a.q + (int64_t)row * a.q_ld + k[0]) = out;
  if ((threadIdx.x & 15) == 0)
    a.scales[(int64_t)g * a.n_rows + row] = bad ? __builtin_nanf("") : top / 448.f;
}

template <typename Row>
void launch_quant(const QuantArgs& a, hipStream_t s) {
  const dim3 grid = flat_grid(((int64_t)a.units + 15) / 16);
  if (a.up)
    hipLaunchKernelGGL((fp8_quant_kernel<Row, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((fp8_quant_kernel<Row, false>), grid, dim3(256), 0, s, a);
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
//
// out[r, n] = sum over blocks b of sx[r, b] sw[n / 128, b] P_b, P_b the sum of
// the block's 128 products of codes: one MFMA (16 weight rows by 16 rows of q,
// K = 128) makes 256 of them, and a fused multiply-add takes each into its fp32
// sum. Weights are the first operand, so a lane's four results are neighbours
// of one out row, whose x scale it needs alone.

struct GemmArgs {
  const uint8_t* w;
  const float* ws;
  const uint8_t* q;
  int64_t q_ld;
  uint32_t q_bytes;           // of q, for its buffer
  const float* qs;            // [KB][q_rows]
  const int32_t* offsets;     // null: one span of every row
  const int32_t* sorted_ids;  // null: row r reads q row r
  void* out;
  int64_t out_ld;
  int32_t q_rows, n_rows, E, N, NT, NB, KB, top_k;
  int32_t n_groups, ks;
};

// One tile: rows row .. end - 1 (as many as the tile takes of them) of expert e, and
// the tile's number among the columns. e < 0: there is none.
struct Span {
  int e, row, end, n;
};

// The spans, cut into tiles of `size` rows. Offsets past the rows count as the last row.
struct Spans {
  const int32_t* offsets;
  int E, n_rows, size;
};
// Four times 64 spans in the lanes of a wave, all of them loaded at once.
struct SpanRows {
  static constexpr int kSpans = 256;
  int lo[4], hi[4];
  __device__ __forceinline__ void load(const Spans& s, int base) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = s.offsets[min(base + 64 * i + lane, s.E)];
      hi[i] = s.offsets[min(base + 64 * i + lane + 1, s.E)];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = min(max(lo[i], 0), s.n_rows);
      hi[i] = base + 64 * i + lane < s.E ? min(max(hi[i], lo[i]), s.n_rows) : lo[i];
    }
  }
  __device__ __forceinline__ int tiles(const Spans& s, int i) const {
    return (hi[i] - lo[i] + s.size - 1) / s.size;
  }
};

// Workgroup `group`'s tile, found by the wave together. The tiles of an XCD (every
// eighth workgroup) are neighbours, an eighth of those that there are, so that they
// share rows and weights in its L2 and no XCD gets more of them.
__device__ __forceinline__ Span find_tile(const int32_t* offsets, int E, int n_rows, int size,
                                          int n_groups, int group) {
  const Spans spans{offsets, E, n_rows, size};
  SpanRows rows;
  int total = (n_rows + size - 1) / size;
  if (offsets) {
    total = 0;
    for (int base = 0; base < E; base += SpanRows::kSpans) {
      rows.load(spans, base);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int sum;
        wave_prefix(rows.tiles(spans, i), &sum);
        total += sum;
      }
    }
  }
  const int per = (int)(((int64_t)total * n_groups + 7) / 8);
  const int64_t at = (int64_t)(group % 8) * per + group / 8;
  if (group / 8 >= per || at >= (int64_t)total * n_groups) return Span{-1, 0, 0, 0};
  int tile = (int)at / n_groups;
  const int n = (int)at - tile * n_groups;
  if (!offsets) return Span{0, tile * size, n_rows, n};
  for (int base = 0; base < E; base += SpanRows::kSpans) {
    if (E > SpanRows::kSpans) rows.load(spans, base);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int sum;
      const int tiles = rows.tiles(spans, i), before = wave_prefix(tiles, &sum);
      if (tile >= 0 && tile < sum) {
        const uint64_t here = __ballot(tile >= before && tile < before + tiles);
        if (!here) return Span{-1, 0, 0, 0};  // sums past 32 bits, of offsets that are none
        const int l = __builtin_ctzll(here);
        const int row = __builtin_amdgcn_readlane(rows.lo[i], l) +
                        (tile - __builtin_amdgcn_readlane(before, l)) * size;
        return Span{base + 64 * i + l, row, __builtin_amdgcn_readlane(rows.hi[i], l), n};
      }
      tile -= sum;
    }
  }
  return Span{-1, 0, 0, 0};
}

// What names the q row that sorted row r reads (r past the rows: the last one's), and
// that q row; -1: none.
__device__ __forceinline__ int source_id(const GemmArgs& a, int r) {
  return a.sorted_ids ? a.sorted_ids[min(r, a.n_rows - 1)] : r;
}
__device__ __forceinline__ int source_row(const GemmArgs& a, int id, int r, int end) {
  const int t = a.sorted_ids ? (int)((uint32_t)id / (uint32_t)a.top_k) : id;
  return r < end && id >= 0 && t < a.q_rows ? t : -1;
}

// A lane's results from column n on, 4 or (a pair of tiles) 8 of them.
template <typename Row, int C>
__device__ __forceinline__ void store_columns(const GemmArgs& a, int64_t row, int n, const float* v) {
  typedef typename Row::elem elem;
  elem* p = static_cast<elem*>(a.out) + row * a.out_ld + n;
  if constexpr (C % Row::kPer16 == 0) {
#pragma unroll
    for (int i = 0; i < C; i += Row::kPer16)
      if (n + i < a.N) store16_any<Row>(p + i, a.N - n - i, Row::narrow16(v + i));
  } else {
    if (n + 4 <= a.N) {
      *reinterpret_cast<u32x2_any*>(p) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (n + i < a.N) p[i] = Row::narrow(v[i]);
    }
  }
}

// A block's products: their sums in fp32, or (FAST, where the route asks for it) as the
// 8-bit instruction makes them.
template <bool FAST>
__device__ __forceinline__ f32x4 block_products(const Fp8Frag& w, const Fp8Frag& q) {
  if constexpr (FAST)
    return mfma_fp8(w, q);
  else
    return mfma_fp8_as_bf16(w, q);
}

// A wave makes 16 columns of 16 rows, operands straight from memory: for calls too
// small to fill the chip with larger tiles. ks waves of a workgroup share a tile's
// blocks and add their sums up in order.
template <typename Row, bool FAST>
__global__ void __launch_bounds__(512) fp8_gemm_stream_kernel(GemmArgs a) {
  __shared__ f32x4 part[8][64];
  const int lane = threadIdx.x & 63, wave = uniform_i32(threadIdx.x >> 6);
  const int nw = (int)(blockDim.x >> 6) / a.ks;
  const Span sp = find_tile(a.offsets, a.E, a.n_rows, 16, a.n_groups, flat_group());
  if (sp.e < 0) return;  // the whole workgroup
  const int kp = wave / nw;
  const int nt = sp.n * nw + wave - kp * nw;
  const bool on = nt < a.NT;
  const int row = sp.row + (lane & 15);
  const int src = source_row(a, source_id(a, row), row, sp.end);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (on) {
    const uint8_t* w =
        a.w + ((int64_t)sp.e * a.NB * 8 * a.KB + fp8_tile(nt, 0, a.KB)) * kFp8Tile + lane * 16;
    const float* ws = a.ws + ((int64_t)sp.e * a.NB + nt / 8) * a.KB;
    const uint8_t* q = a.q + (int64_t)max(src, 0) * a.q_ld + (lane >> 4) * 32;
    const float* qs = a.qs + max(src, 0);
    const int k0 = a.KB * kp / a.ks, k1 = a.KB * (kp + 1) / a.ks;
    for (int kb = k0; kb < k1; ++kb) {
      const Fp8Frag wf = load_frag(w + (int64_t)kb * (8 * kFp8Tile), 1024);
      const Fp8Frag qf = load_frag(q + kb * 128, 16);
      const float s = ws[kb] * qs[(int64_t)kb * a.q_rows];
      const f32x4 p = block_products<FAST>(wf, qf);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] = fmaf(p[v], s, acc[v]);
    }
  }
  if (a.ks > 1) {
    part[wave][lane] = acc;
    __syncthreads();
    if (kp > 0) return;
    for (int j = 1; j < a.ks; ++j) acc += part[wave + j * nw][lane];
  }
  if (on && src >= 0) {
    const float v[4] = {acc[0], acc[1], acc[2], acc[3]};
    store_columns<Row, 4>(a, row, fp8_column(nt, lane >> 4), v);
  }
}

// The same for spans of many rows: a workgroup of WM by WN waves makes a tile of
// BM rows by BN columns, a wave MT by NT pieces of 16 by 16 of it. The blocks go
// through LDS stages, two of rows and WS of weights: while one is multiplied the next is
// on its way, the weights' (which are read from farthest) up to two blocks ahead, moved by
// loads that write LDS themselves. Weights lie there as they are packed; a q row's
// eight 16-byte pieces change places by the row's number (piece p of row r holds k
// piece p ^ (r / 2 % 8)), so that 8 lanes read one row whole and the 16 rows of an
// operand come from all 64 banks.
//
// 8192 rows of 4096 by 4096 x 4096 take 244 to 251 us with fp32 sums, in tiles of 128 x
// 128 (198 at the rate of the library's bf16 product). With fast sums, in tiles of 256 x
// 256, they take 124 to 140, by the card's power (2.0 to 2.2 PFLOP/s; a library's product
// of E4M3 with one scale: 102 us on one of them): the clock falls to 1.85 GHz, and a block
// takes 3280 cycles of which the matrix instructions fill 2048, the rest being the next
// block's latency. The rest of this is of fast sums too. The third stage of weights, all
// that 160 KB of LDS have room for, took spans of 256 rows and 1024 columns from 129 to
// 122 us. Where in a block it is requested, and which waves go first, made no difference;
// touching the lines of later blocks early cost 10% and more, as a CU's requests are near
// their limit. Of many spans a tile's start counts as well: its span and its rows' numbers
// in one round trip each, shared through LDS, took 32768 rows of 128 experts from 129 to
// 119 us, rows past a span's end that ask for nothing and are not multiplied to 110 (by
// chance half of the spans have a tile of a few rows). Workgroups that stay and ask for
// the next tile's first block before they store won where tiles are alike (138 -> 137 us
// of the first case) and lost more where they are not (2048 x 4096 weights: 196 -> 218),
// as they cannot take over from each other.
template <int WM, int WN, int MT, int NT, int WS>
struct Tile {
  static constexpr int W = WM * WN, BM = WM * MT * 16, BN = WN * NT * 16;
  static constexpr int kW = BN * 128, kX = BM * 128;  // bytes of a stage
  static constexpr int kLds = WS * kW + 2 * kX;
  static constexpr int kWLoads = BN / 8 / W, kXLoads = BM / 8 / W;  // of 1 KB, a wave's
};

// The offset in q of a row that is not there: behind its end, where loads give zeros
// without a request.
constexpr uint32_t kNoRow = 0xffff8000u;

// 16 bytes of each lane straight into LDS, lane l's at p + 16 l.
__device__ __forceinline__ void to_lds(rsrc_t r, uint32_t lane_off, uint32_t off, uint8_t* p) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)p, 16,
                                           lane_off, off, 0, 0);
}

// One block of 128 k of a wave's pieces from a stage. The matrix instructions of one
// column of pieces are issued between the multiply-adds of the column before, which
// would wait for their results otherwise.
template <bool FAST, int MT, int NT>
__device__ __forceinline__ void tile_block(const uint8_t* w, const uint8_t* x, int lane,
                                           const float (&s)[MT], f32x4 (&acc)[MT][NT]) {
  const int row = lane & 15, piece = (lane >> 4) * 2;
  Fp8Frag xf[MT], wf[2];
  wf[0] = load_frag(w + lane * 16, 1024);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xf[i].h[h] = *reinterpret_cast<const u32x4*>(x + (i * 16 + row) * 128 +
                                                   ((piece + h) ^ ((row >> 1) & 7)) * 16);
  f32x4 d[2][MT];
#pragma unroll
  for (int j = 0; j <= NT; ++j) {
    __builtin_amdgcn_sched_barrier(0);
    if (j + 1 < NT) wf[(j + 1) & 1] = load_frag(w + (j + 1) * kFp8Tile + lane * 16, 1024);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (j < NT) d[j & 1][i] = block_products<FAST>(wf[j & 1], xf[i]);
      if (j > 0) {
#pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[i][j - 1][v] = fmaf(d[(j - 1) & 1][i][v], s[i], acc[i][j - 1][v]);
      }
    }
    if constexpr (FAST) {
      if (j + 1 < NT) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // LDS reads
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (j < NT) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
        if (j > 0) __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);   // VALU
      }
    }
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <typename Row, bool FAST, int WM, int WN, int MT, int NT, int WS>
__global__ void __launch_bounds__(64 * WM * WN, 2) fp8_gemm_tile_kernel(GemmArgs a) {
  typedef Tile<WM, WN, MT, NT, WS> T;
  extern __shared__ __attribute__((aligned(16))) uint8_t stages[];  // of weights, then of rows
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform_i32(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const Span sp = find_tile(a.offsets, a.E, a.n_rows, T::BM, a.n_groups, flat_group());
  if (sp.e < 0) return;  // the whole workgroup
  const int n0 = sp.n * (T::BN / 16);  // in tiles of 16 columns

  // the rows' q rows, one a thread, where the second block's rows go later
  uint8_t* const x_stages = stages + WS * T::kW;
  int* const source = reinterpret_cast<int*>(x_stages + T::kX);
  if (tid < T::BM) source[tid] = source_row(a, source_id(a, sp.row + tid), sp.row + tid, sp.end);
  __syncthreads();

  // what this wave moves: its share of the weights' and of the rows' kilobytes
  const int first = n0 / 8;  // block of 128 columns
  const uint32_t slab = (uint32_t)a.KB * (8 * kFp8Tile);  // bytes of one
  const int blocks = min(a.NB - first, (T::BN + 127) / 128);
  const rsrc_t w_buf = buffer(a.w + ((int64_t)sp.e * a.NB + first) * slab, blocks * slab);
  uint32_t w_off[T::kWLoads];  // of columns past the last block: that block's again
#pragma unroll
  for (int i = 0; i < T::kWLoads; ++i) {
    const int c = wave * T::kWLoads + i, nt = n0 % 8 + c / 2;
    w_off[i] = min(nt / 8, blocks - 1) * slab + (nt % 8) * kFp8Tile + (c & 1) * 1024;
  }
  const rsrc_t x_buf = buffer(a.q, a.q_bytes);
  const rsrc_t s_buf = buffer(a.qs, (uint32_t)a.KB * (uint32_t)a.q_rows * 4);
  uint32_t x_off[T::kXLoads];
#pragma unroll
  for (int i = 0; i < T::kXLoads; ++i) {
    const int r = (wave * T::kXLoads + i) * 8 + (lane >> 3), src = source[r];
    x_off[i] = src < 0 ? kNoRow : (uint32_t)src * (uint32_t)a.q_ld;
    asm volatile("" : "+v"(x_off[i]));  // else the sum takes two registers
    x_off[i] += ((lane & 7) ^ ((r >> 1) & 7)) * 16;
  }
  uint32_t s_off[MT], there = 0;  // a bit for each of the pieces' rows that there are
  float xs[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int src = source[(wm * MT + i) * 16 + (lane & 15)];
    s_off[i] = 4u * max(src, 0);
    there |= (src >= 0 ? 1u : 0u) << i;
  }
  const float* w_scale =
      a.ws + ((int64_t)sp.e * a.NB + min((n0 + wn * NT) / 8, a.NB - 1)) * a.KB;
  float ws = 0.f;
  // past the last block, the last one again (into stages that nothing reads)
  auto request_w = [&](int kb, int at) {
    kb = min(kb, a.KB - 1);
#pragma unroll
    for (int i = 0; i < T::kWLoads; ++i)
      to_lds(w_buf, lane * 16, w_off[i] + kb * (8 * kFp8Tile),
             stages + at * T::kW + (wave * T::kWLoads + i) * 1024);
  };
  auto request_x = [&](int kb) {
    uint8_t* p = x_stages + (kb & 1) * T::kX;
    kb = min(kb, a.KB - 1);
#pragma unroll
    for (int i = 0; i < T::kXLoads; ++i)
      to_lds(x_buf, x_off[i], kb * 128, p + (wave * T::kXLoads + i) * 1024);
#pragma unroll
    for (int i = 0; i < MT; ++i)
      xs[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          s_buf, s_off[i], (uint32_t)kb * (uint32_t)a.q_rows * 4, 0));
    ws = w_scale[kb];
  };
  f32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // a wave without rows leaves its matrix unit to the others. With fp32 sums the branch
  // costs as much as it saves (one weight, as above, 249 -> 259 us; 32768 skewed rows of 128
  // experts 153 -> 149).
  const bool live = !FAST || sp.row + wm * MT * 16 < sp.end;
  request_w(0, 0);
  request_x(0);
  __builtin_amdgcn_sched_barrier(0);  // the weights that need not be there are the last loads
  if (WS == 3) request_w(1, 1);
  int at = 0;  // the weights' stage
  for (int kb = 0; kb < a.KB; ++kb) {
    wait_loads<(WS - 2) * T::kWLoads>();
    stage_barrier();  // block kb has arrived, and the stages to be filled are no longer read
    float s[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) s[i] = xs[i] * ws;
    request_x(kb + 1);
    __builtin_amdgcn_sched_barrier(0);
    request_w(kb + WS - 1, at == 0 ? WS - 1 : at - 1);
    if (live)
      tile_block<FAST, MT, NT>(stages + at * T::kW + wn * NT * kFp8Tile,
                              x_stages + (kb & 1) * T::kX + wm * MT * 16 * 128, lane, s, acc);
    at = at == WS - 1 ? 0 : at + 1;
  }
  wait_loads<0>();  // the stages are another workgroup's next
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int row = sp.row + (wm * MT + i) * 16 + (lane & 15);
    if (!(there >> i & 1)) continue;
#pragma unroll
    for (int j = 0; j < NT; j += 2) {
      float v[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) v[c] = acc[i][j + c / 4][c % 4];
      store_columns<Row, 8>(a, row, fp8_column(n0 + wn * NT + j, lane >> 4), v);
    }
  }
}

// Sums of fewer than 2^31 tiles, so that a tile's number is an int.
constexpr int64_t kMaxTiles = 0x7f000000ll;

// Tiles of `size` rows that the spans can have: each of a span's but the last is full.
int64_t most_tiles(const GemmArgs& a, int size) {
  if (!a.offsets) return ((int64_t)a.n_rows + size - 1) / size;
  return (int64_t)a.n_rows / size + std::min(a.E, a.n_rows);
}

template <typename Row, bool FAST, int WM, int WN, int MT, int NT, int WS>
int32_t launch_tile(const char* who, GemmArgs a, hipStream_t s) {
  typedef Tile<WM, WN, MT, NT, WS> T;
  const int64_t m_tiles = most_tiles(a, T::BM);
  a.n_groups = (a.NT * 16 + T::BN - 1) / T::BN;
  if (m_tiles * a.n_groups > kMaxTiles)
    return fail(MLORA_ERR_INVALID, "%s: too many rows for one call", who);
  hipLaunchKernelGGL((fp8_gemm_tile_kernel<Row, FAST, WM, WN, MT, NT, WS>),
                     flat_grid(m_tiles * a.n_groups + 7), dim3(64 * T::W), T::kLds, s, a);
  return launch_status(who);
}

template <typename Row, bool FAST>
int32_t launch_stream(const char* who, GemmArgs a, hipStream_t s) {
  const int64_t m_tiles = most_tiles(a, 16);
  a.ks = 1;
  while (a.ks < 8 && a.ks * 2 <= a.KB && m_tiles * a.NT * a.ks < 2048) a.ks *= 2;
  const int waves = std::max(4, a.ks);
  a.n_groups = (a.NT + waves / a.ks - 1) / (waves / a.ks);
  if (m_tiles * a.n_groups > kMaxTiles)
    return fail(MLORA_ERR_INVALID, "%s: too many rows for one call", who);
  hipLaunchKernelGGL((fp8_gemm_stream_kernel<Row, FAST>), flat_grid(m_tiles * a.n_groups + 7),
                     dim3(64 * waves), 0, s, a);
  return launch_status(who);
}

template <typename Row, bool FAST>
int32_t launch_gemm(const char* who, const GemmArgs& a, hipStream_t s) {
  const Fp8Form form = plan_fp8(a.n_rows, a.E, a.N, FAST);
  if (form == kFp8Stream) return launch_stream<Row, FAST>(who, a, s);
  if constexpr (FAST)
    if (form == kFp8Rows256) return launch_tile<Row, FAST, 4, 2, 4, 8, 3>(who, a, s);
  if (form == kFp8Rows128) return launch_tile<Row, FAST, 2, 2, 4, 4, 2>(who, a, s);
  if (form == kFp8Rows64) return launch_tile<Row, FAST, 2, 2, 2, 4, 2>(who, a, s);
  return launch_tile<Row, FAST, 1, 4, 2, 2, 2>(who, a, s);
}

int64_t blocks_of(int32_t v) { return ((int64_t)v + 127) / 128; }

// Sizes of a route, or why they are refused.
int32_t check_sizes(const char* who, int32_t n_experts, int32_t k_in, int32_t n_out) {
  if (n_experts < 1 || n_experts > kFp8MaxExperts)
    return fail(MLORA_ERR_INVALID, "%s: n_experts=%d outside [1, %d]", who, n_experts,
                kFp8MaxExperts);
  if (k_in < 1 || k_in > kFp8MaxDim || n_out < 1 || n_out > kFp8MaxDim)
    return fail(MLORA_ERR_INVALID, "%s: k_in=%d, n_out=%d outside [1, %d]", who, k_in, n_out,
                kFp8MaxDim);
  if (n_experts * blocks_of(k_in) * blocks_of(n_out) > kMaxRows)
    return fail(MLORA_ERR_INVALID, "%s: %d experts of %d x %d are too large", who, n_experts, n_out,
                k_in);
  return MLORA_OK;
}

}  // namespace

int32_t check_fp8_route(const char* who, const char* name, const mlora_fp8_route* r) {
  if (!r) return fail(MLORA_ERR_INVALID, "%s: NULL %s route", who, name);
  if (int32_t rc = check_sizes(who, r->n_experts, r->k_in, r->n_out)) return rc;
  if (!r->weights || !r->scales || !aligned(r->weights, 16) || !aligned(r->scales, 4))
    return fail(MLORA_ERR_INVALID, "%s: %s route without packed weights", who, name);
  if (r->fast_sums != 0 && r->fast_sums != 1)
    return fail(MLORA_ERR_INVALID, "%s: %s route's fast_sums=%d is neither 0 nor 1", who, name,
                r->fast_sums);
  return MLORA_OK;
}

}  // namespace mlora

using namespace mlora;

extern "C" int32_t mlora_fp8_row_width(int32_t k) {
  // an odd number of blocks: rows a multiple of 512 bytes apart would come from few
  // of an L2's 16 channels of 256 bytes
  return k < 1 || k > kFp8MaxDim ? 0 : (int32_t)((blocks_of(k) | 1) * 128);
}

extern "C" uint64_t mlora_fp8_packed_bytes(int32_t n_experts, int32_t k_in, int32_t n_out) {
  if (check_sizes("mlora_fp8_packed_bytes", n_experts, k_in, n_out)) return 0;
  const uint64_t blocks = (uint64_t)n_experts * blocks_of(k_in) * blocks_of(n_out);
  return blocks * (8 * kFp8Tile) + ((blocks * 4 + 255) / 256) * 256;
}

extern "C" int32_t mlora_fp8_pack(const uint8_t* w, const float* scales, int32_t n_experts,
                                  int32_t k_in, int32_t n_out, int32_t transpose, void* packed,
                                  uint64_t packed_bytes, mlora_fp8_route* route, void* stream) {
  const char* who = "mlora_fp8_pack";
  if (int32_t rc = check_sizes(who, n_experts, k_in, n_out)) return rc;
  if (!w || !scales || !packed || !route) return fail(MLORA_ERR_INVALID, "%s: NULL pointer", who);
  if (!aligned(packed, 256))
    return fail(MLORA_ERR_INVALID, "%s: packed must be 256-byte aligned", who);
  const uint64_t need = mlora_fp8_packed_bytes(n_experts, k_in, n_out);
  if (packed_bytes < need)
    return fail(MLORA_ERR_CAPACITY, "%s: packed of %llu bytes, %llu needed", who,
                (unsigned long long)packed_bytes, (unsigned long long)need);
  Fp8PackArgs a{};
  a.w = w;
  a.scales = scales;
  a.N = n_out;
  a.K = k_in;
  a.NB = (int32_t)blocks_of(n_out);
  a.KB = (int32_t)blocks_of(k_in);
  a.cells = (int64_t)n_experts * a.NB * a.KB;
  a.packed = static_cast<uint8_t*>(packed);
  a.packed_scales = reinterpret_cast<float*>(a.packed + a.cells * (8 * kFp8Tile));
  a.transpose = transpose != 0;
  (void)hipGetLastError();
  hipLaunchKernelGGL(fp8_pack_kernel, flat_grid(a.cells), dim3(256), 0,
                     reinterpret_cast<hipStream_t>(stream), a);
  if (int32_t rc = launch_status(who)) return rc;
  route->weights = a.packed;
  route->scales = a.packed_scales;
  route->n_experts = n_experts;
  route->k_in = k_in;
  route->n_out = n_out;
  route->fast_sums = 0;
  return MLORA_OK;
}

extern "C" int32_t mlora_fp8_quant(const void* x, int64_t x_ld, const void* up, int64_t up_ld,
                                   int32_t dtype, int64_t n_rows, int32_t k, uint8_t* q,
                                   int64_t q_ld, float* q_scales, void* stream) {
  const char* who = "mlora_fp8_quant";
  if (dtype != MLORA_BF16 && dtype != MLORA_F32)
    return fail(MLORA_ERR_INVALID, "%s: dtype %d is neither bf16 nor f32", who, dtype);
  if (n_rows < 0 || n_rows > kMaxRows)
    return fail(MLORA_ERR_INVALID, "%s: n_rows=%lld out of range", who, (long long)n_rows);
  if (k < 1 || k > kFp8MaxDim)
    return fail(MLORA_ERR_INVALID, "%s: k=%d outside [1, %d]", who, k, kFp8MaxDim);
  if (x_ld < k || (up && up_ld < k))
    return fail(MLORA_ERR_INVALID, "%s: row stride below k=%d", who, k);
  if (q_ld < mlora_fp8_row_width(k) || q_ld % 16 != 0)
    return fail(MLORA_ERR_INVALID, "%s: q row stride %lld is not a multiple of 16 from %d on", who,
                (long long)q_ld, mlora_fp8_row_width(k));
  if (n_rows == 0) {
    clear_error();
    return MLORA_OK;
  }
  if (!x || !q || !q_scales) return fail(MLORA_ERR_INVALID, "%s: NULL pointer", who);
  if (!aligned(q, 16)) return fail(MLORA_ERR_INVALID, "%s: q must be 16-byte aligned", who);
  QuantArgs a{};
  a.x = x;
  a.x_ld = x_ld;
  a.up = up;
  a.up_ld = up_ld;
  a.q = q;
  a.q_ld = q_ld;
  a.scales = q_scales;
  a.n_rows = (int32_t)n_rows;
  a.K = k;
  a.groups = (int32_t)blocks_of(k);
  if (n_rows * a.groups > 0xf0000000ll)
    return fail(MLORA_ERR_INVALID, "%s: too many rows for one call", who);
  a.units = (uint32_t)(n_rows * a.groups);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (dtype == MLORA_BF16)
    launch_quant<Bf16Row>(a, s);
  else
    launch_quant<F32Row>(a, s);
  return launch_status(who);
}

extern "C" int32_t mlora_fp8_gemm(const mlora_fp8_route* route, const uint8_t* q, int64_t q_rows,
                                  int64_t q_ld, const float* q_scales, void* out, int64_t out_ld,
                                  int32_t out_dtype, int64_t n_rows,
                                  const int32_t* expert_offsets, const int32_t* sorted_ids,
                                  int32_t top_k, void* stream) {
  const char* who = "mlora_fp8_gemm";
  if (int32_t rc = check_fp8_route(who, "weight", route)) return rc;
  if (out_dtype != MLORA_BF16 && out_dtype != MLORA_F32)
    return fail(MLORA_ERR_INVALID, "%s: dtype %d is neither bf16 nor f32", who, out_dtype);
  if (n_rows < 0 || n_rows > kMaxRows || q_rows < 0 || q_rows > kMaxRows)
    return fail(MLORA_ERR_INVALID, "%s: n_rows=%lld or q_rows=%lld out of range", who,
                (long long)n_rows, (long long)q_rows);
  if (top_k < 1 || top_k > kFp8MaxExperts)
    return fail(MLORA_ERR_INVALID, "%s: top_k=%d outside [1, %d]", who, top_k, kFp8MaxExperts);
  if (!expert_offsets && route->n_experts != 1)
    return fail(MLORA_ERR_INVALID, "%s: no expert_offsets for %d experts", who, route->n_experts);
  if (!sorted_ids && q_rows < n_rows)
    return fail(MLORA_ERR_INVALID, "%s: q_rows=%lld below n_rows=%lld", who, (long long)q_rows,
                (long long)n_rows);
  if (q_ld < mlora_fp8_row_width(route->k_in) || q_ld % 16 != 0)
    return fail(MLORA_ERR_INVALID, "%s: q row stride %lld is not a multiple of 16 from %d on", who,
                (long long)q_ld, mlora_fp8_row_width(route->k_in));
  if (out_ld < route->n_out)
    return fail(MLORA_ERR_INVALID, "%s: out row stride %lld below n_out=%d", who,
                (long long)out_ld, route->n_out);
  if (n_rows == 0 || q_rows == 0) {
    clear_error();
    return MLORA_OK;
  }
  if (!q || !q_scales || !out) return fail(MLORA_ERR_INVALID, "%s: NULL pointer", who);
  if (!aligned(q, 16)) return fail(MLORA_ERR_INVALID, "%s: q must be 16-byte aligned", who);
  const int64_t width = mlora_fp8_row_width(route->k_in);
  if (q_ld > kNoRow || (q_rows - 1) * q_ld + width > kNoRow)
    return fail(MLORA_ERR_INVALID, "%s: q spans 4 GiB or nearly; split the call", who);
  GemmArgs a{};
  a.q_bytes = (uint32_t)((q_rows - 1) * q_ld + width);
  a.w = static_cast<const uint8_t*>(route->weights);
  a.ws = static_cast<const float*>(route->scales);
  a.q = q;
  a.q_ld = q_ld;
  a.qs = q_scales;
  a.offsets = expert_offsets;
  a.sorted_ids = sorted_ids;
  a.out = out;
  a.out_ld = out_ld;
  a.q_rows = (int32_t)q_rows;
  a.n_rows = (int32_t)n_rows;
  a.E = route->n_experts;
  a.N = route->n_out;
  a.NT = fp8_tiles(route->n_out);
  a.NB = (int32_t)blocks_of(route->n_out);
  a.KB = (int32_t)blocks_of(route->k_in);
  a.top_k = top_k;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (out_dtype == MLORA_F32) return launch_gemm<F32Row, false>(who, a, s);
  return route->fast_sums ? launch_gemm<Bf16Row, true>(who, a, s)
                          : launch_gemm<Bf16Row, false>(who, a, s);
}
