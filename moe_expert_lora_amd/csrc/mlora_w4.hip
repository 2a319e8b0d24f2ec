// Products with 4-bit expert weights for gfx950 (MI355X): the base projection
// of the rows the fold adds its deltas to, for decode batches.
//
//     out[r, n] = sum_k x[src(r), k] * (q[e(r), n, k] - z[e, n, k / group])
//                                    * s[e, n, k / group]
//
// The products run on bf16 MFMA (16x16x32). A 4-bit value v is put into the
// mantissa of a bf16 as 16 + v (one and/or per pair of values, exact), so a
// lane's 8 values take 7 VALU operations; the group's offset 16 + z comes off
// in fp32 afterwards, with the group's sum of x, which one more MFMA per k
// step (a constant first operand) leaves in every lane. Each group's partial
// product is scaled in fp32, so weights are never rounded. fp32 rows are split
// into three bf16 parts (8 + 8 + 8 bits, exact), one MFMA each: the products
// stay exact and the sums fp32.
//
// The offset makes |16 + v| sums cancel: their fp32 rounding is about 5 times
// that of a plain sum of the same length, far below one bf16 rounding and
// below 1e-6 of an fp32 result. A row of x with an infinity or a NaN gives
// NaN outputs for that row alone.
//
// Work: a workgroup owns one expert and NT column tiles of 16; its waves split
// k in chunks of 128 and add their sums up through LDS in wave order. Each
// workgroup finds its expert's rows by scanning the ids (decode batches: a few
// KB, from L2), takes them 16 at a time as the second MFMA operand straight
// from x, and streams its weights once per 16 rows.
#include <type_traits>

#include "mlora_device.h"

namespace mlora {
namespace {

typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int kMaxW4Experts = 1024;
constexpr uint32_t kMaxBuf = 0xFFFFFF00u;  // largest range one buffer resource describes
constexpr uint32_t kPast = 0xFFFFFFF0u;    // an offset past every buffer: the load gives 0
constexpr int kScan = 2048;                // rows scanned (and listed) at a time
constexpr int kMaxWaves = 8;

__device__ __forceinline__ rsrc_t buf(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 ld16(rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Packed layout. Weights: per expert and column tile of 16, ksteps = ceil(k /
// 32) steps of 256 bytes. Four steps make a chunk of 1024 bytes in which lane l
// of a wave finds its 16 bytes at 16 l: word i is step i, column l % 16, k
// values 32 i + 8 (l / 16) .. + 7. The steps after the last whole chunk lie
// one after the other, lane l's word at 4 l. In a word, values 2p and 2p + 1
// of the 8 sit at bits 3 + 4p and 19 + 4p (p = 3 wraps round at bit 31), so
// that a shift (a rotation for p = 3), a mask and an or leave the two bf16
// values 16 + v side by side.
// Scales and zero points: per expert, tile and scale block (the groups of one
// chunk, or the chunks of one group), lane group l / 16 finds SG groups of 4
// columns each; a zero point is kept as the byte 16 + z.
struct W4Layout {
  int64_t tiles, ksteps, blocks, sg, tile_bytes;
  int64_t w_bytes, s_bytes, z_bytes, s_off, z_off, total;
};

W4Layout w4_layout(int64_t E, int64_t K, int64_t N, int64_t group, int es, bool zeros) {
  W4Layout l;
  l.tiles = (N + 15) / 16;
  l.ksteps = (K + 31) / 32;
  l.sg = group < 128 ? 128 / group : 1;
  const int64_t span = group < 128 ? 128 : group;
  l.blocks = (K + span - 1) / span;
  l.tile_bytes = l.ksteps * 256;
  l.w_bytes = E * l.tiles * l.tile_bytes;
  l.s_bytes = E * l.tiles * l.blocks * 16 * l.sg * es;
  l.z_bytes = zeros ? E * l.tiles * l.blocks * 16 * l.sg : 0;
  l.s_off = (l.w_bytes + 255) & ~255ll;
  l.z_off = (l.s_off + l.s_bytes + 255) & ~255ll;
  l.total = (l.z_off + l.z_bytes + 255) & ~255ll;
  return l;
}

struct W4PackArgs {
  const uint8_t* q;
  const void* scales;
  const uint8_t* zeros;
  uint32_t* w;
  void* s;
  uint8_t* z;
  int64_t words, cells;
  int32_t K, N, group, groups, tiles, ksteps, blocks, sg;
};

// One thread per packed word, then one per scale cell.
template <typename Row>
__global__ void __launch_bounds__(256) w4_pack_kernel(W4PackArgs a) {
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at < a.words) {
    const int64_t per_tile = (int64_t)a.ksteps * 64;
    const int64_t et = at / per_tile;
    const int w = (int)(at - et * per_tile);
    const int whole = a.ksteps / 4 * 256;  // words of the tile in whole chunks
    int step, lane;
    if (w < whole) {
      step = w / 256 * 4 + (w & 3);
      lane = (w & 255) >> 2;
    } else {
      step = a.ksteps / 4 * 4 + (w - whole) / 64;
      lane = (w - whole) & 63;
    }
    const int64_t e = et / a.tiles;
    const int n = (int)(et - e * a.tiles) * 16 + (lane & 15);
    const int k = step * 32 + (lane >> 4) * 8;
    uint32_t out = 0;
    if (n < a.N && k < a.K) {
      const uint8_t* p = a.q + ((e * a.N + n) * (int64_t)a.K + k) / 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t b = p[i];
        out |= (b & 15) << (3 + 4 * i);
        const uint32_t hi = b >> 4;
        out |= i < 3 ? hi << (19 + 4 * i) : (hi << 31) | (hi >> 1);
      }
    }
    a.w[at] = out;
    return;
  }
  const int64_t c = at - a.words;
  if (c >= a.cells) return;
  // cell: [expert][tile][block][lane group][sg][4 columns]
  const int col = (int)(c & 3);
  int64_t rest = c >> 2;
  const int sg = (int)(rest % a.sg);
  rest /= a.sg;
  const int lg = (int)(rest & 3);
  rest >>= 2;
  const int blk = (int)(rest % a.blocks);
  rest /= a.blocks;
  const int64_t e = rest / a.tiles;
  const int n = (int)(rest - e * a.tiles) * 16 + lg * 4 + col;
  const int g = blk * a.sg + sg;
  typedef typename Row::elem elem;
  const bool in = n < a.N && g < a.groups;
  const int64_t src = (e * a.N + n) * a.groups + g;
  static_cast<elem*>(a.s)[c] = in ? static_cast<const elem*>(a.scales)[src] : (elem)0;
  if (a.z) a.z[c] = (uint8_t)(16 + (in ? (a.zeros[src] & 15) : 0));
}

struct W4Args {
  const uint8_t* w;
  const uint8_t* s;
  const uint8_t* z;
  const void* x;
  void* out;
  const int32_t* ids;
  int64_t out_ld;
  int64_t tile_bytes;
  uint32_t x_bytes;
  uint32_t x_ld_bytes;
  uint32_t topk;          // rows per x row (1: a row of its own)
  int32_t n_rows;
  int32_t E;              // 0: no ids, one weight
  int32_t K, N;
  int32_t tiles, ksteps, blocks, per_block;  // per_block: chunks per scale block
  int32_t slices;
  int32_t out_vec;        // rows of out start on 4 elements
};

// 8 packed values of one column -> the bf16 values 16 + v.
__device__ __forceinline__ u32x4 unpack(uint32_t w) {
  constexpr uint32_t kMask = 0x00780078u, kBase = 0x41804180u;
  u32x4 r;
  r[0] = (w & kMask) | kBase;
  r[1] = ((w >> 4) & kMask) | kBase;
  r[2] = ((w >> 8) & kMask) | kBase;
  r[3] = (__builtin_amdgcn_alignbit(w, w, 12) & kMask) | kBase;
  return r;
}

// Second MFMA operand of one k step: bf16 as loaded, or an fp32 row's three
// bf16 parts, smallest first.
template <bool F32>
struct XFrag {
  static constexpr int kParts = F32 ? 3 : 1;
  u32x4 p[kParts];
};

template <bool F32>
__device__ __forceinline__ XFrag<F32> load_x(rsrc_t rx, uint32_t row_off, int k, int K) {
  XFrag<F32> f;
  const bool in = row_off != kPast && k < K;
  if constexpr (!F32) {
    f.p[0] = ld16(rx, in ? row_off + (uint32_t)k * 2u : kPast);
  } else {
    const uint32_t off = row_off + (uint32_t)k * 4u;
    const u32x4 a = ld16(rx, in ? off : kPast), b = ld16(rx, in ? off + 16u : kPast);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v0 = __uint_as_float(i < 2 ? a[2 * i] : b[2 * i - 4]);
      const float v1 = __uint_as_float(i < 2 ? a[2 * i + 1] : b[2 * i - 3]);
      const uint32_t h = pack_bf16(v0, v1);
      const float r0 = v0 - lo_f(h), r1 = v1 - hi_f(h);
      const uint32_t m = pack_bf16(r0, r1);
      f.p[2][i] = h;
      f.p[1][i] = m;
      f.p[0][i] = pack_bf16(r0 - lo_f(m), r1 - hi_f(m));
    }
  }
  return f;
}

template <bool F32, int SG, bool ZP, int NT>
__global__ void __launch_bounds__(64 * kMaxWaves) w4_kernel(W4Args a) {
  typedef typename std::conditional<F32, F32Row, Bf16Row>::type Row;
  constexpr int kEs = F32 ? 4 : 2;
  constexpr int kCols = 16 * NT, kStride = kCols + 4;
  __shared__ int list[kScan];
  __shared__ int counts[kMaxWaves];
  extern __shared__ float red[];  // [waves][16][kStride]
  const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, lg = lane >> 4;
  const int waves = (int)(blockDim.x >> 6), wave = uniform_i32(tid >> 6);
  const int e = (int)blockIdx.x / a.slices;
  const int tile0 = ((int)blockIdx.x - e * a.slices) * NT;
  const int n0 = tile0 * 16;
  typename Row::elem* out = static_cast<typename Row::elem*>(a.out);
  const rsrc_t rx = buf(a.x, a.x_bytes);
  const int64_t et0 = (int64_t)e * a.tiles + tile0;
  const int chunks = (a.ksteps + 3) >> 2, whole = a.ksteps >> 2;
  constexpr float kZero = ZP ? -1.f : -24.f;
  const uint32_t kc = pack_bf16(kZero, kZero);
  const u32x4 cons = {kc, kc, kc, kc};

  for (int seg = 0; seg < a.n_rows; seg += kScan) {
    const int len = min(kScan, a.n_rows - seg);
    int n_list = len;
    if (a.E > 0) {
      if (seg > 0) __syncthreads();
      // Each wave scans a run of 64 * rounds ids and lists its hits behind
      // those of the waves before it: in row order, so that workgroups which
      // share an expert's rows agree on the list.
      const int rounds = (len + 64 * waves - 1) / (64 * waves);  // <= 32
      const int first = wave * rounds * 64 + lane;
      uint32_t hits = 0;
      int n_wave = 0;
      for (int r = 0; r < rounds; ++r) {
        const int i = first + r * 64;
        const int id = i < len ? a.ids[seg + i] : -1;
        // workgroups of the place after the last expert write the zeros of
        // rows without one
        const bool hit = i < len && ((uint32_t)id < (uint32_t)a.E ? id : a.E) == e;
        n_wave += __popcll(__ballot(hit));
        hits |= (hit ? 1u : 0u) << r;
      }
      if (lane == 0) counts[wave] = n_wave;
      __syncthreads();
      int at = 0;
      n_list = 0;
      for (int w = 0; w < waves; ++w) {
        at += w < wave ? counts[w] : 0;
        n_list += counts[w];
      }
      at = uniform_i32(at);
      n_list = uniform_i32(n_list);
      for (int r = 0; r < rounds; ++r) {
        const bool hit = (hits >> r) & 1;
        const uint64_t m = __ballot(hit);
        if (hit)
          list[at + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                              __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u))] =
              seg + first + r * 64;
        at += __popcll(m);
      }
      __syncthreads();
      if (e == a.E) {
        const int all = (int)(blockDim.x * gridDim.y);
        for (int i = tid + (int)(blockIdx.y * blockDim.x); i < n_list * kCols; i += all) {
          const int n = n0 + i % kCols;
          if (n < a.N) out[(int64_t)list[i / kCols] * a.out_ld + n] = 0;
        }
        continue;
      }
    }
    for (int b0 = (int)blockIdx.y * 16; b0 < n_list; b0 += (int)gridDim.y * 16) {
      const int at = b0 + li;
      const int row = at < n_list ? (a.E > 0 ? list[at] : seg + at) : -1;
      const uint32_t row_off = row >= 0 ? (uint32_t)row / a.topk * a.x_ld_bytes : kPast;
      f32x4 acc[NT] = {};
      for (int c = wave; c < chunks; c += waves) {
        u32x4 w[NT];
        uint32_t sw[NT][SG * kEs];  // 4 scales per group: 2 or 4 words
        uint32_t zw[NT][SG];
        const int blk = c / a.per_block;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // tiles past the last read the last one again and are not stored
          const int64_t et = et0 + min(nt, a.tiles - 1 - tile0);
          const uint8_t* p = a.w + et * a.tile_bytes + (int64_t)c * 1024;
          if (c < whole) {
            w[nt] = *reinterpret_cast<const u32x4*>(p + lane * 16);
          } else {
            const int left = a.ksteps & 3;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[nt][i] = i < left ? *reinterpret_cast<const uint32_t*>(p + i * 256 + lane * 4) : 0;
          }
          const int64_t cell = ((et * a.blocks + blk) * 4 + lg) * SG;
          const uint32_t* ps = reinterpret_cast<const uint32_t*>(a.s + cell * 4 * kEs);
#pragma unroll
          for (int i = 0; i < SG * kEs; ++i) sw[nt][i] = ps[i];
          if constexpr (ZP) {
            const uint32_t* pz = reinterpret_cast<const uint32_t*>(a.z + cell * 4);
#pragma unroll
            for (int i = 0; i < SG; ++i) zw[nt][i] = pz[i];
          }
        }
        XFrag<F32> x[4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          x[ks] = load_x<F32>(rx, row_off, c * 128 + ks * 32 + lg * 8, a.K);
#pragma unroll
        for (int sg = 0; sg < SG; ++sg) {
          constexpr int kPer = 4 / SG;
          f32x4 dc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ks = sg * kPer; ks < (sg + 1) * kPer; ++ks)
#pragma unroll
            for (int p = 0; p < XFrag<F32>::kParts; ++p) dc = mfma(cons, x[ks].p[p], dc);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            f32x4 s = ZP ? f32x4{0.f, 0.f, 0.f, 0.f} : dc;
#pragma unroll
            for (int ks = sg * kPer; ks < (sg + 1) * kPer; ++ks) {
              const u32x4 wf = unpack(w[nt][ks]);
#pragma unroll
              for (int p = 0; p < XFrag<F32>::kParts; ++p) s = mfma(wf, x[ks].p[p], s);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float t = s[i];
              if constexpr (ZP)
                t = fmaf((float)((zw[nt][sg] >> (8 * i)) & 0xffu), dc[i], t);
              float sc;
              if constexpr (F32)
                sc = __uint_as_float(sw[nt][sg * 4 + i]);
              else
                sc = (i & 1) ? hi_f(sw[nt][sg * 2 + i / 2]) : lo_f(sw[nt][sg * 2 + i / 2]);
              acc[nt][i] = fmaf(sc, t, acc[nt][i]);
            }
          }
        }
      }
      // the waves' sums, added in wave order
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<f32x4*>(&red[(wave * 16 + li) * kStride + nt * 16 + lg * 4]) = acc[nt];
      __syncthreads();
      for (int i = tid; i < 16 * kCols / 4; i += (int)blockDim.x) {
        const int r = i / (kCols / 4), c4 = i % (kCols / 4) * 4;
        f32x4 sum = *reinterpret_cast<const f32x4*>(&red[r * kStride + c4]);
        for (int w = 1; w < waves; ++w)
          sum += *reinterpret_cast<const f32x4*>(&red[(w * 16 + r) * kStride + c4]);
        const int n = n0 + c4;
        if (b0 + r >= n_list || n >= a.N) continue;
        const int orow = a.E > 0 ? list[b0 + r] : seg + b0 + r;
        typename Row::elem* o = out + (int64_t)orow * a.out_ld + n;
        if (a.out_vec && n + 4 <= a.N) {
          if constexpr (F32)
            *reinterpret_cast<f32x4*>(o) = sum;
          else
            *reinterpret_cast<u32x2*>(o) =
                u32x2{pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < a.N) o[j] = Row::narrow(sum[j]);
        }
      }
      __syncthreads();
    }
  }
}

struct W4Plan {
  int nt, waves, splits;
};

W4Plan plan_w4(const mlora_w4_route* r, int64_t n_rows, int64_t experts) {
  W4Plan p;
  const int64_t tiles = (r->n_out + 15) / 16, chunks = (r->k_in + 127) / 128;
  // Column tiles per workgroup: 4 while that leaves 512 workgroups or more,
  // else 1, so that a single weight is spread over as many CUs as it has tiles.
  p.nt = experts * ((tiles + 3) / 4) >= 512 ? 4 : 1;
  // Waves: one per chunk up to 8, and no more than it takes for the fewest
  // chunks per wave.
  const int64_t per = (chunks + kMaxWaves - 1) / kMaxWaves;
  p.waves = (int)((chunks + per - 1) / per);
  // Rows of one expert over several workgroups once an expert holds more than
  // two blocks of 16 on average.
  const int64_t blocks = (n_rows + experts * 16 - 1) / (experts * 16);
  p.splits = (int)(blocks <= 2 ? 1 : blocks > 64 ? 32 : (blocks + 1) / 2);
  return p;
}

template <bool F32, int SG, bool ZP>
void launch_w4(const W4Args& a0, const W4Plan& p, int64_t places, hipStream_t s) {
  W4Args a = a0;
  a.slices = (a.tiles + p.nt - 1) / p.nt;
  const dim3 grid((unsigned)(places * a.slices), (unsigned)p.splits), block(64 * p.waves);
  const size_t lds = (size_t)p.waves * 16 * (16 * p.nt + 4) * 4;
  if (p.nt == 4)
    hipLaunchKernelGGL((w4_kernel<F32, SG, ZP, 4>), grid, block, lds, s, a);
  else
    hipLaunchKernelGGL((w4_kernel<F32, SG, ZP, 1>), grid, block, lds, s, a);
}

template <bool F32>
void dispatch_w4(const W4Args& a, const W4Plan& p, int sg, int64_t places, hipStream_t s) {
  if (a.z) {
    if (sg == 4) return launch_w4<F32, 4, true>(a, p, places, s);
    if (sg == 2) return launch_w4<F32, 2, true>(a, p, places, s);
    return launch_w4<F32, 1, true>(a, p, places, s);
  }
  if (sg == 4) return launch_w4<F32, 4, false>(a, p, places, s);
  if (sg == 2) return launch_w4<F32, 2, false>(a, p, places, s);
  launch_w4<F32, 1, false>(a, p, places, s);
}

int32_t check_w4(const char* who, int32_t E, int32_t K, int32_t N, int32_t group,
                 int32_t dtype) {
  if (dtype != MLORA_BF16 && dtype != MLORA_F32)
    return fail(MLORA_ERR_INVALID, "%s: dtype %d is neither bf16 nor f32", who, dtype);
  if (E < 1 || E > kMaxW4Experts)
    return fail(MLORA_ERR_INVALID, "%s: n_experts=%d outside [1, %d]", who, E, kMaxW4Experts);
  if (K < 8 || K % 8 != 0 || K > (1 << 20))
    return fail(MLORA_ERR_INVALID, "%s: k_in=%d must be a multiple of 8 in [8, 2^20]", who, K);
  if (N < 1 || N > (1 << 20))
    return fail(MLORA_ERR_INVALID, "%s: n_out=%d outside [1, 2^20]", who, N);
  if (group != 32 && group != 64 && (group < 128 || group % 128 != 0))
    return fail(MLORA_ERR_INVALID, "%s: group=%d must be 32, 64 or a multiple of 128", who, group);
  return MLORA_OK;
}

}  // namespace
}  // namespace mlora

using namespace mlora;

extern "C" uint64_t mlora_w4_packed_bytes(int32_t n_experts, int32_t k_in, int32_t n_out,
                                          int32_t group, int32_t dtype, int32_t has_zeros) {
  if (check_w4("mlora_w4_packed_bytes", n_experts, k_in, n_out, group, dtype) != MLORA_OK)
    return 0;
  clear_error();
  return (uint64_t)w4_layout(n_experts, k_in, n_out, group, dtype == MLORA_BF16 ? 2 : 4,
                             has_zeros != 0)
      .total;
}

extern "C" int32_t mlora_w4_pack(const uint8_t* q, const void* scales, const uint8_t* zeros,
                                 int32_t n_experts, int32_t k_in, int32_t n_out, int32_t group,
                                 int32_t dtype, void* packed, uint64_t packed_bytes,
                                 mlora_w4_route* route, void* stream) {
  const char* who = "mlora_w4_pack";
  if (int32_t rc = check_w4(who, n_experts, k_in, n_out, group, dtype)) return rc;
  if (!q || !scales || !packed || !route)
    return fail(MLORA_ERR_INVALID, "%s: NULL pointer", who);
  if (!aligned(packed, 256))
    return fail(MLORA_ERR_INVALID, "%s: packed must be 256-byte aligned", who);
  const W4Layout l = w4_layout(n_experts, k_in, n_out, group, dtype == MLORA_BF16 ? 2 : 4,
                               zeros != nullptr);
  if (packed_bytes < (uint64_t)l.total)
    return fail(MLORA_ERR_CAPACITY, "%s: packed of %llu bytes, %lld needed", who,
                (unsigned long long)packed_bytes, (long long)l.total);
  W4PackArgs a{};
  uint8_t* base = static_cast<uint8_t*>(packed);
  a.q = q;
  a.scales = scales;
  a.zeros = zeros;
  a.w = reinterpret_cast<uint32_t*>(base);
  a.s = base + l.s_off;
  a.z = zeros ? base + l.z_off : nullptr;
  a.words = l.w_bytes / 4;
  a.cells = (int64_t)n_experts * l.tiles * l.blocks * 16 * l.sg;
  a.K = k_in;
  a.N = n_out;
  a.group = group;
  a.groups = (k_in + group - 1) / group;
  a.tiles = (int32_t)l.tiles;
  a.ksteps = (int32_t)l.ksteps;
  a.blocks = (int32_t)l.blocks;
  a.sg = (int32_t)l.sg;
  const int64_t grid = (a.words + a.cells + 255) / 256;
  if (grid > 0x7fffffffll) return fail(MLORA_ERR_INVALID, "%s: weights too large", who);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (dtype == MLORA_BF16)
    hipLaunchKernelGGL(w4_pack_kernel<Bf16Row>, dim3((unsigned)grid), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(w4_pack_kernel<F32Row>, dim3((unsigned)grid), dim3(256), 0, s, a);
  if (int32_t rc = launch_status(who)) return rc;
  route->weights = a.w;
  route->scales = a.s;
  route->zeros = a.z;
  route->n_experts = n_experts;
  route->k_in = k_in;
  route->n_out = n_out;
  route->group = group;
  route->dtype = dtype;
  return MLORA_OK;
}

extern "C" int32_t mlora_w4_gather_gemv(const mlora_w4_route* route, const void* x,
                                        int64_t x_rows, int64_t x_ld, int32_t x_by_row, void* out,
                                        int64_t out_ld, const int32_t* ids, int64_t n_rows,
                                        int32_t top_k, void* stream) {
  const char* who = "mlora_w4_gather_gemv";
  if (!route) return fail(MLORA_ERR_INVALID, "%s: NULL route", who);
  if (int32_t rc = check_w4(who, route->n_experts, route->k_in, route->n_out, route->group,
                            route->dtype))
    return rc;
  if (!ids && route->n_experts != 1)
    return fail(MLORA_ERR_INVALID, "%s: a route of %d experts needs ids", who, route->n_experts);
  if (top_k < 1) return fail(MLORA_ERR_INVALID, "%s: top_k=%d must be positive", who, top_k);
  if (n_rows < 0 || n_rows > kMaxRows)
    return fail(MLORA_ERR_INVALID, "%s: n_rows=%lld out of range", who, (long long)n_rows);
  const int64_t need = x_by_row ? n_rows : (n_rows + top_k - 1) / top_k;
  if (x_rows < need || x_rows > kMaxRows)
    return fail(MLORA_ERR_INVALID, "%s: %lld x rows, need >= %lld", who, (long long)x_rows,
                (long long)need);
  const int es = route->dtype == MLORA_BF16 ? 2 : 4;
  if (x_ld < route->k_in || x_ld % 8 != 0)
    return fail(MLORA_ERR_INVALID, "%s: x_ld=%lld must be a multiple of 8, >= k_in=%d", who,
                (long long)x_ld, route->k_in);
  if (out_ld < route->n_out)
    return fail(MLORA_ERR_INVALID, "%s: out_ld=%lld below n_out=%d", who, (long long)out_ld,
                route->n_out);
  if (n_rows == 0) {
    clear_error();
    return MLORA_OK;
  }
  if (!x || !out || !route->weights || !route->scales)
    return fail(MLORA_ERR_INVALID, "%s: NULL device pointer", who);
  if (!aligned(x, 16)) return fail(MLORA_ERR_INVALID, "%s: x must be 16-byte aligned", who);
  // the rows the call reads (views into wider tensors end at k_in)
  if (x_ld > (int64_t)kMaxBuf / es ||
      (need - 1) * x_ld + route->k_in > (int64_t)kMaxBuf / es)
    return fail(MLORA_ERR_INVALID, "%s: x exceeds 4 GiB", who);
  const W4Layout l = w4_layout(route->n_experts, route->k_in, route->n_out, route->group, es,
                               route->zeros != nullptr);
  W4Args a{};
  a.w = static_cast<const uint8_t*>(route->weights);
  a.s = static_cast<const uint8_t*>(route->scales);
  a.z = static_cast<const uint8_t*>(route->zeros);
  a.x = x;
  a.out = out;
  a.ids = ids;
  a.out_ld = out_ld;
  a.tile_bytes = l.tile_bytes;
  a.x_bytes = (uint32_t)(((need - 1) * x_ld + route->k_in) * es);
  a.x_ld_bytes = (uint32_t)(x_ld * es);
  a.topk = x_by_row ? 1u : (uint32_t)top_k;
  a.n_rows = (int32_t)n_rows;
  a.E = ids ? route->n_experts : 0;
  a.K = route->k_in;
  a.N = route->n_out;
  a.tiles = (int32_t)l.tiles;
  a.ksteps = (int32_t)l.ksteps;
  a.blocks = (int32_t)l.blocks;
  a.per_block = route->group <= 128 ? 1 : route->group / 128;
  a.out_vec = out_ld % 4 == 0 && aligned(out, 4 * es);
  const int64_t places = ids ? route->n_experts + 1 : 1;
  const W4Plan p = plan_w4(route, n_rows, route->n_experts);
  if (places * ((l.tiles + p.nt - 1) / p.nt) > 0x3fffffffll)
    return fail(MLORA_ERR_INVALID, "%s: weights too large for one launch", who);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (route->dtype == MLORA_BF16)
    dispatch_w4<false>(a, p, (int)l.sg, places, s);
  else
    dispatch_w4<true>(a, p, (int)l.sg, places, s);
  return launch_status(who);
}
