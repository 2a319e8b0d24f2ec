// Products with 8-bit floating-point expert weights (OCP E4M3, a scale for each
// block of 128 x 128), for gfx950 (MI355X): the weights' layout, the rows'
// quantiser, and the product over rows sorted by expert.
#include "mlora_fp8.h"

namespace mlora {
namespace {

// ---------------------------------------------------------------------------
// pack
// ---------------------------------------------------------------------------
//
// A thread moves the 16 bytes of one lane and half (mlora_fp8.h). Forward, they
// lie together in the source row; transposed, they are 16 rows of one column,
// and 16 lanes of a wave read neighbouring columns.

struct Fp8PackArgs {
  const uint8_t* w;
  const float* scales;
  uint8_t* packed;
  float* packed_scales;
  int64_t chunks, cells;  // 16-byte pieces of the weights, scales
  int32_t N, K, NB, KB;   // of the packed (transposed) matrix
  int32_t transpose;
};

__global__ void __launch_bounds__(256) fp8_pack_kernel(Fp8PackArgs a) {
  int64_t i = (int64_t)flat_group() * 256 + threadIdx.x;
  if (i < a.chunks) {
    const int lane = (int)(i & 63), half = (int)(i >> 6) & 1;
    int64_t t = i >> 7;
    const int kb = (int)(t % a.KB);
    t /= a.KB;
    const int nt = (int)(t % (a.NB * 8));
    const int64_t e = t / (a.NB * 8);
    const int n = nt * 16 + (lane & 15), k = kb * 128 + (lane >> 4) * 32 + half * 16;
    const uint8_t* src = a.w + e * a.N * a.K;
    u32x4 v = {0, 0, 0, 0};
    if (n < a.N && k < a.K) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (k + j < a.K) {
          const uint32_t b = a.transpose ? src[(int64_t)(k + j) * a.N + n] : src[(int64_t)n * a.K + k + j];
          v[j / 4] |= b << (8 * (j % 4));
        }
      }
    }
    *reinterpret_cast<u32x4*>(a.packed + i * 16) = v;
    return;
  }
  i -= a.chunks;
  if (i < a.cells) {
    const int kb = (int)(i % a.KB);
    const int64_t t = i / a.KB;
    const int nb = (int)(t % a.NB);
    const int64_t e = t / a.NB;
    a.packed_scales[i] = a.scales[e * a.NB * a.KB + (a.transpose ? (int64_t)kb * a.NB + nb
                                                                 : (int64_t)nb * a.KB + kb)];
  }
}

// ---------------------------------------------------------------------------
// quantise rows
// ---------------------------------------------------------------------------
//
// A group of 128 values of a row: m = its largest magnitude (448 * 2^-126 at
// least), scale = m / 448, code = 448 x / m to the nearest E4M3 value, ties to
// even. 16 lanes hold a group, 8 values each. The quotient is exact to one
// rounding: with e the exponent of m, both 448 x 2^-e (exact for a bf16 x) and
// m 2^-e in [1, 2) are fp32 values, and a quotient by the rounded reciprocal,
// corrected once by its remainder, is the correctly rounded one; a bf16 x and m
// have 8 bits each, so a quotient that is not half way between two codes stays
// off that border by more than fp32's rounding. An fp32 x is divided in fp64,
// and what the rounding to fp32 cut off is kept in its last bit, so that the
// codes are those of the exact quotient too. silu(x) up is rounded to fp32 first.
// A group with an infinity or NaN gets a NaN as scale and codes of 0.

struct QuantArgs {
  const void* x;
  int64_t x_ld;
  const void* up;  // null: x itself
  int64_t up_ld;
  uint8_t* q;
  int64_t q_ld;
  float* scales;   // [groups][n_rows]
  int64_t units;   // n_rows * groups
  int32_t n_rows, K, groups;
};

// Four E4M3 codes, the first in the low byte.
__device__ __forceinline__ uint32_t pack_fp8(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return (uint32_t)v;
}

template <typename Row, bool SILU, bool WIDE>
__global__ void __launch_bounds__(256) fp8_quant_kernel(QuantArgs a) {
  const int64_t unit = (int64_t)flat_group() * 16 + (threadIdx.x >> 4);
  if (unit >= a.units) return;  // whole rows of 16 lanes: the reduction stays in them
  const int row = (int)(unit / a.groups);
  const int g = (int)(unit - (int64_t)row * a.groups);
  const int k = g * 128 + (threadIdx.x & 15) * 8;
  float v[8];
  load8<Row, WIDE>(a.x, (int64_t)row * a.x_ld, k, a.K, v);
  if constexpr (SILU) {
    float u[8];
    load8<Row, WIDE>(a.up, (int64_t)row * a.up_ld, k, a.K, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] / (1.f + expf(-v[i])) * u[i];
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  m = group_max<16>(m);
  const bool bad = m >= 0x7f800000u;
  m = bad ? 0x3f800000u : max(m, 0x04e00000u);  // 448 * 2^-126 = 1.75 * 2^-118
  const float top = __uint_as_float(m);
  float c[8];
  if constexpr (sizeof(typename Row::elem) == 4 && !SILU) {
    const double r = 1.0 / (double)top;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double t = (double)v[i] * 448.0 * r;
      const float f = (float)t;
      // an even last bit with something cut off: one step towards it
      const double off = t - (double)f;
      const uint32_t b = __float_as_uint(f);
      const bool odd = (b & 1u) || fabs(off) <= fabs(t) * 0x1p-40;
      const bool grow = (off > 0.0) == (f > 0.f);
      c[i] = odd || f == 0.f ? f : __uint_as_float(grow ? b + 1u : b - 1u);
    }
  } else {
    const int e = (int)(m >> 23) - 127;
    const float den = __uint_as_float((m & 0x7fffffu) | 0x3f800000u);
    const float num = ldexpf(448.f, -e);
    const float r = 1.f / den;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = v[i] * num;
      const float q = t * r;
      c[i] = fmaf(fmaf(-q, den, t), r, q);
    }
  }
  u32x2 out = {pack_fp8(c[0], c[1], c[2], c[3]), pack_fp8(c[4], c[5], c[6], c[7])};
  if (bad) out = u32x2{0, 0};
  *reinterpret_cast<u32x2*>(a.q + (int64_t)row * a.q_ld + k) = out;
  if ((threadIdx.x & 15) == 0)
    a.scales[(int64_t)g * a.n_rows + row] = bad ? __builtin_nanf("") : top / 448.f;
}

template <typename Row, bool SILU>
void launch_quant(const QuantArgs& a, bool wide, hipStream_t s) {
  const dim3 grid = flat_grid((a.units + 15) / 16);
  if (wide)
    hipLaunchKernelGGL((fp8_quant_kernel<Row, SILU, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((fp8_quant_kernel<Row, SILU, false>), grid, dim3(256), 0, s, a);
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
  const float* qs;            // [KB][q_rows]
  const int32_t* offsets;     // null: one span of every row
  const int32_t* sorted_ids;  // null: row r reads q row r
  void* out;
  int64_t out_ld;
  int32_t q_rows, n_rows, E, N, NT, NB, KB, top_k;
  int32_t n_groups, ks;
};

// The rows of one tile: up to `size` of expert e from `row` on, below `end`.
struct Span {
  int e, row, end;
};

// Tile number `tile` among the spans' tiles of `size` rows, found by the wave
// together: 64 spans at a time, their tiles' prefix in the lanes. e < 0: there
// are fewer tiles. Offsets past the rows count as the last row.
__device__ __forceinline__ Span find_tile(const int32_t* offsets, int E, int n_rows, int size,
                                          int tile) {
  if (!offsets) {
    const int row = tile * size;
    return Span{row < n_rows ? 0 : -1, row, n_rows};
  }
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < E; base += 64) {
    const int e = base + lane;
    int lo = 0, hi = 0;
    if (e < E) {
      lo = min(max(offsets[e], 0), n_rows);
      hi = min(max(offsets[e + 1], lo), n_rows);
    }
    const int tiles = (hi - lo + size - 1) / size;
    int sum;
    const int before = wave_prefix(tiles, &sum);
    if (tile < sum) {
      const uint64_t here = __ballot(tile >= before && tile < before + tiles);
      const int l = __builtin_ctzll(here);
      const int row = __builtin_amdgcn_readlane(lo, l) +
                      (tile - __builtin_amdgcn_readlane(before, l)) * size;
      return Span{base + l, row, __builtin_amdgcn_readlane(hi, l)};
    }
    tile -= sum;
  }
  return Span{-1, 0, 0};
}

// The q row that sorted row r reads; -1: none.
__device__ __forceinline__ int source_row(const GemmArgs& a, int r, int end) {
  if (r >= end) return -1;
  if (!a.sorted_ids) return r < a.q_rows ? r : -1;
  const int id = a.sorted_ids[r];
  const int t = (int)((uint32_t)id / (uint32_t)a.top_k);
  return id >= 0 && t < a.q_rows ? t : -1;
}

template <typename Row>
__device__ __forceinline__ void store4(const GemmArgs& a, int64_t row, int n, f32x4 v, bool wide) {
  typename Row::elem* p = static_cast<typename Row::elem*>(a.out) + row * a.out_ld + n;
  if (wide && n + 4 <= a.N) {
    if constexpr (sizeof(typename Row::elem) == 2)
      *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    else
      *reinterpret_cast<f32x4*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < a.N) p[i] = Row::narrow(v[i]);
  }
}

// A block's products, as exact as the result's type asks for.
template <typename Row>
__device__ __forceinline__ f32x4 block_products(const Fp8Frag& w, const Fp8Frag& q) {
  if constexpr (sizeof(typename Row::elem) == 2)
    return mfma_fp8(w, q);
  else
    return mfma_fp8_as_bf16(w, q);
}

// A wave makes 16 columns of 16 rows, operands straight from memory; ks waves
// of a workgroup share a tile's blocks and add their sums up in order.
template <typename Row>
__global__ void __launch_bounds__(512) fp8_gemm_stream_kernel(GemmArgs a, bool wide) {
  __shared__ f32x4 part[8][64];
  const int lane = threadIdx.x & 63, wave = uniform_i32(threadIdx.x >> 6);
  const int nw = (int)(blockDim.x >> 6) / a.ks;
  const int group = flat_group();
  const Span sp = find_tile(a.offsets, a.E, a.n_rows, 16, group / a.n_groups);
  if (sp.e < 0) return;  // the whole workgroup
  const int kp = wave / nw;
  const int nt = (group % a.n_groups) * nw + wave - kp * nw;
  const bool on = nt < a.NT;
  const int row = sp.row + (lane & 15);
  const int src = source_row(a, row, sp.end);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (on) {
    const uint8_t* w = a.w + (((int64_t)sp.e * a.NB * 8 + nt) * a.KB) * kFp8Tile + lane * 16;
    const float* ws = a.ws + ((int64_t)sp.e * a.NB + nt / 8) * a.KB;
    const uint8_t* q = a.q + (int64_t)max(src, 0) * a.q_ld + (lane >> 4) * 32;
    const float* qs = a.qs + max(src, 0);
    const int k0 = a.KB * kp / a.ks, k1 = a.KB * (kp + 1) / a.ks;
    for (int kb = k0; kb < k1; ++kb) {
      const Fp8Frag wf = load_frag(w + (int64_t)kb * kFp8Tile, 1024);
      const Fp8Frag qf = load_frag(q + kb * 128, 16);
      const float s = ws[kb] * qs[(int64_t)kb * a.q_rows];
      const f32x4 p = block_products<Row>(wf, qf);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(p[i], s, acc[i]);
    }
  }
  if (a.ks > 1) {
    part[wave][lane] = acc;
    __syncthreads();
    if (kp > 0) return;
    for (int j = 1; j < a.ks; ++j) acc += part[wave + j * nw][lane];
  }
  if (on && src >= 0) store4<Row>(a, row, nt * 16 + (lane >> 4) * 4, acc, wide);
}

// Sums of fewer than 2^31 tiles, so that a tile's number is an int.
constexpr int64_t kMaxTiles = 0x7f000000ll;

template <typename Row>
int32_t launch_gemm(const char* who, GemmArgs a, bool wide, hipStream_t s) {
  const int64_t m_tiles = (int64_t)a.n_rows / 16 + std::min(a.E, a.n_rows);
  a.ks = 1;
  while (a.ks < 8 && a.ks * 2 <= a.KB && m_tiles * a.NT * a.ks < 2048) a.ks *= 2;
  const int waves = std::max(4, a.ks);
  a.n_groups = (a.NT + waves / a.ks - 1) / (waves / a.ks);
  if (m_tiles * a.n_groups > kMaxTiles)
    return fail(MLORA_ERR_INVALID, "%s: too many rows for one call", who);
  hipLaunchKernelGGL((fp8_gemm_stream_kernel<Row>), flat_grid(m_tiles * a.n_groups),
                     dim3(64 * waves), 0, s, a, wide);
  return launch_status(who);
}

// Sizes of a route, or why they are refused.
int32_t check_sizes(const char* who, int32_t n_experts, int32_t k_in, int32_t n_out) {
  if (n_experts < 1 || n_experts > kFp8MaxExperts)
    return fail(MLORA_ERR_INVALID, "%s: n_experts=%d outside [1, %d]", who, n_experts,
                kFp8MaxExperts);
  if (k_in < 1 || k_in > kFp8MaxDim || n_out < 1 || n_out > kFp8MaxDim)
    return fail(MLORA_ERR_INVALID, "%s: k_in=%d, n_out=%d outside [1, %d]", who, k_in, n_out,
                kFp8MaxDim);
  return MLORA_OK;
}

int64_t blocks_of(int32_t v) { return ((int64_t)v + 127) / 128; }

}  // namespace

int32_t check_fp8_route(const char* who, const char* name, const mlora_fp8_route* r) {
  if (!r) return fail(MLORA_ERR_INVALID, "%s: NULL %s route", who, name);
  if (int32_t rc = check_sizes(who, r->n_experts, r->k_in, r->n_out)) return rc;
  if (!r->weights || !r->scales || !aligned(r->weights, 16) || !aligned(r->scales, 4))
    return fail(MLORA_ERR_INVALID, "%s: %s route without packed weights", who, name);
  return MLORA_OK;
}

}  // namespace mlora

using namespace mlora;

extern "C" int32_t mlora_fp8_row_width(int32_t k) {
  return k < 1 || k > kFp8MaxDim ? 0 : (int32_t)(blocks_of(k) * 128);
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
  a.chunks = a.cells * (8 * kFp8Tile / 16);
  a.packed = static_cast<uint8_t*>(packed);
  a.packed_scales = reinterpret_cast<float*>(a.packed + a.chunks * 16);
  a.transpose = transpose != 0;
  const int64_t groups = (a.chunks + a.cells + 255) / 256;
  if (groups > kMaxRows) return fail(MLORA_ERR_INVALID, "%s: weights too large", who);
  (void)hipGetLastError();
  hipLaunchKernelGGL(fp8_pack_kernel, flat_grid(groups), dim3(256), 0,
                     reinterpret_cast<hipStream_t>(stream), a);
  if (int32_t rc = launch_status(who)) return rc;
  route->weights = a.packed;
  route->scales = a.packed_scales;
  route->n_experts = n_experts;
  route->k_in = k_in;
  route->n_out = n_out;
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
  a.units = n_rows * a.groups;
  if ((a.units + 15) / 16 > kMaxTiles)
    return fail(MLORA_ERR_INVALID, "%s: too many rows for one call", who);
  const int64_t per = dtype == MLORA_BF16 ? 8 : 4;
  const bool wide = k % 8 == 0 && x_ld % per == 0 && aligned(x, 16) &&
                    (!up || (up_ld % per == 0 && aligned(up, 16)));
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (dtype == MLORA_BF16) {
    if (up)
      launch_quant<Bf16Row, true>(a, wide, s);
    else
      launch_quant<Bf16Row, false>(a, wide, s);
  } else {
    if (up)
      launch_quant<F32Row, true>(a, wide, s);
    else
      launch_quant<F32Row, false>(a, wide, s);
  }
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
  GemmArgs a{};
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
  a.NT = (route->n_out + 15) / 16;
  a.NB = (int32_t)blocks_of(route->n_out);
  a.KB = (int32_t)blocks_of(route->k_in);
  a.top_k = top_k;
  const bool wide = out_ld % 4 == 0 && aligned(out, out_dtype == MLORA_BF16 ? 8 : 16);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  return out_dtype == MLORA_BF16 ? launch_gemm<Bf16Row>(who, a, wide, s)
                                 : launch_gemm<F32Row>(who, a, wide, s);
}
