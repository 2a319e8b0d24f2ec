// Products with 4-bit expert weights for gfx950 (MI355X): the base projection
// of the rows the fold adds its deltas to, for decode batches.
//
//     out[r, n] = sum_k x[src(r), k] * (q[e(r), n, k] - z[e, n, k / group])
//                                    * s[e, n, k / group]
//
// The products run on bf16 MFMA (16x16x32): 16 rows of x by 16 columns of
// weights. A 4-bit value v is packed as sign and magnitude of 2 v - 15, an odd
// number whose lowest bit is not kept. As the byte s000mmm1 that is the fp8
// (e4m3) number (2 v - 15) / 512, below 2^-5 where those lie evenly, and the
// conversion to bf16 with a scale of 256 makes the exact v - 7.5 of it: a lane's
// 8 values take 7 VALU operations. A group's sums start at -(z - 7.5) times the
// group's sum of x, so that v - z is what they hold at its end; they are then
// scaled in fp32, so weights are never rounded. A lane's values are of one
// column: one scale and one zero point for all of them. fp32 rows are split into
// three bf16 parts (8 + 8 + 8 bits, exact while the last is no subnormal number,
// from |x| = 2^-103), one MFMA each: the products stay exact and the sums fp32.
// Up to |x| = 2^117 no sum overflows: one of a group of at most 128 values stays
// below (7.5 + 7.5) sum |x|.
//
// The offset is small (0.5 without zero points), so that the sums, like a plain
// fp32 one's, pass through little that cancels: relative L2 errors of fp32 rows of
// 264 and 768 values, means 0 and 3, are 0.9 to 3.3 u (u = 2^-24), a plain fp32
// sum's 0.8 to 1.6. (With bf16 values 16 + v, made by an and/or a pair, they were 5.7
// to 39 u, in about the same time: 128 experts of 768 x 2048, 640 rows 21.7 us, as
// now, of 2048 x 768, 2048 rows 30.7, now 31.0.)
// A row of x with an infinity or a NaN gives no finite outputs, in that row alone.
//
// Two forms, each of which reads an expert's weights once per 16 or 32 of its
// rows. Every workgroup finds its expert's rows by scanning the ids (decode
// batches: a few KB, from L2). The split form, for few column tiles, has a
// workgroup own one or two tiles, its waves split k and x rows go straight to the
// operands. The streaming form stages x rows in LDS once per workgroup and gives
// each wave whole pairs of tiles.
//
// What bounds them, at 128 experts of 2048 x 768, groups of 128, bf16 rows: one row
// each on average 21 us a call, 5 rows 24.7, 16 rows 30 (fp32 rows, three products
// and three reads of x from LDS for one: 24.8, 32.3, 56.5); the main loop reads
// weights at 6.3 TB/s, as fast as a CU's cache takes misses on (32 KB on their way,
// 1.4 us each).
// Ahead of it lie 8 to 10 us in which the ids, then x arrive, one round trip after
// the other, and only the first weights beside them. Single weights of a few MB:
// those round trips and the launch (2048 x 2048, one row: 4.3 us).
#include <type_traits>

#include "mlora_device.h"
#include "mlora_w4_plan.h"

namespace mlora {
namespace {

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxW4Experts = 1024;
constexpr uint32_t kMaxBuf = 0xFFFFFF00u;  // largest range one buffer resource describes
constexpr uint32_t kPast = 0xFFFFFF40u;    // an offset past every buffer: the load gives 0
constexpr int kNT = 2;                     // non-temporal: weights are read once

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

// Packed layout. Weights: per expert and pair of column tiles of 16, ksteps =
// ceil(k / 32) steps of 2 x 256 bytes. Four steps make a chunk of 2 x 1024 bytes,
// one tile behind the other, in which lane l of a wave finds its 16 bytes at
// 16 l: word i is step i, column l % 16, k values 32 i + 8 (l / 16) .. + 7. A last
// chunk of fewer steps keeps as many words per lane; a lane still loads 16 bytes
// there, and what it reads of the words behind meets x values of 0. In a word,
// value i < 4 has its sign at bit 7 of byte i and its magnitude (without the lowest
// bit) at bits 3:1; value 4 + i has its sign at bit 0 of byte 3 - i and its
// magnitude at bits 6:4, lowest bit first, so that the word reversed holds values
// 4 to 7 as the word itself holds 0 to 3.
// Scales and zero points: per expert, pair and scale block (the groups of one
// chunk, or the chunks of one group), column l % 16 finds SG groups of the two
// tiles' values; a zero point is a byte.
struct W4Layout {
  int64_t pairs, ksteps, blocks, sg;
  int64_t w_bytes, s_bytes, z_bytes, s_off, z_off, total;
};

W4Layout w4_layout(int64_t E, int64_t K, int64_t N, int64_t group, int es, bool zeros) {
  W4Layout l;
  l.pairs = (N + 31) / 32;
  l.ksteps = (K + 31) / 32;
  l.sg = group < 128 ? 128 / group : 1;
  const int64_t span = group < 128 ? 128 : group;
  l.blocks = (K + span - 1) / span;
  l.w_bytes = E * l.pairs * l.ksteps * 512;
  l.s_bytes = E * l.pairs * l.blocks * 32 * l.sg * es;
  l.z_bytes = zeros ? E * l.pairs * l.blocks * 32 * l.sg : 0;
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
  int32_t K, N, group, groups, pairs, ksteps, blocks, sg;
};

// One thread per packed word, then one per scale cell.
template <typename Row>
__global__ void __launch_bounds__(256) w4_pack_kernel(W4PackArgs a) {
  const int64_t at = (int64_t)flat_group() * 256 + threadIdx.x;
  if (at < a.words) {
    const int64_t per_pair = (int64_t)a.ksteps * 128;
    const int64_t ep = at / per_pair;
    const int w = (int)(at - ep * per_pair);
    const int whole = a.ksteps / 4 * 512;  // words of the pair in whole chunks
    int step, lane, tile;
    if (w < whole) {
      step = w / 512 * 4 + (w & 3);
      tile = (w >> 8) & 1;
      lane = (w & 255) >> 2;
    } else {
      const int left = a.ksteps & 3, r = w - whole;
      tile = r / (left * 64);
      step = a.ksteps / 4 * 4 + r % left;
      lane = r / left & 63;
    }
    const int64_t e = ep / a.pairs;
    const int n = (int)(ep - e * a.pairs) * 32 + tile * 16 + (lane & 15);
    const int k = step * 32 + (lane >> 4) * 8;
    uint32_t out = 0;
    if (n < a.N && k < a.K) {
      const uint8_t* p = a.q + ((e * a.N + n) * (int64_t)a.K + k) / 2;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t v = p[i / 2] >> (4 * (i & 1)) & 15;
        // 2 v - 15 = +- (2 m + 1)
        const uint32_t sign = v < 8, m = (v & 7) ^ (sign ? 7u : 0u);
        const uint32_t byte = sign << 7 | m << 1;
        out |= i < 4 ? byte << (8 * i) : __builtin_bitreverse32(byte << (8 * (i - 4)));
      }
    }
    a.w[at] = out;
    return;
  }
  const int64_t c = at - a.words;
  if (c >= a.cells) return;
  // cell: [expert][pair][block][16 columns][sg][2 tiles]
  const int tile = (int)(c & 1);
  int64_t rest = c >> 1;
  const int sg = (int)(rest % a.sg);
  rest /= a.sg;
  const int col = (int)(rest & 15);
  rest >>= 4;
  const int blk = (int)(rest % a.blocks);
  rest /= a.blocks;
  const int64_t e = rest / a.pairs;
  const int n = (int)(rest - e * a.pairs) * 32 + tile * 16 + col;
  const int g = blk * a.sg + sg;
  typedef typename Row::elem elem;
  const bool in = n < a.N && g < a.groups;
  const int64_t src = (e * a.N + n) * a.groups + g;
  static_cast<elem*>(a.s)[c] = in ? static_cast<const elem*>(a.scales)[src] : (elem)0;
  if (a.z) a.z[c] = in ? (uint8_t)(a.zeros[src] & 15) : (uint8_t)0;
}

struct W4Args {
  const uint8_t* w;
  const uint8_t* s;
  const uint8_t* z;
  const void* x;
  void* out;
  int64_t out_ld;
  uint32_t x_bytes;
  uint32_t x_ld_bytes;
  uint32_t topk;          // rows per x row (1: a row of its own)
  uint32_t topk_magic;    // floor((2^32 - 1) / topk)
  int32_t K, N;
  int32_t ksteps, blocks;
  uint32_t block_magic;   // ceil(2^31 / chunks per scale block)
  int32_t pairs, per_slice;  // tile pairs; streaming form: those of a slice
  int32_t pair_waves;     // pairs a workgroup's waves hold at a time
  uint32_t wave_magic;    // ceil(2^32 / pair_waves)
  int32_t turns;          // ring places of a pair, per wave
  int32_t panel, panel_turns;   // chunks of x in LDS, and their places per wave
  int32_t out_vec;        // rows of out start on 4 elements
};

// What a kernel's start needs. These lead its arguments as plain values, which
// arrive in registers; the struct lies in memory, three cold lines away.
struct W4Lead {
  const int32_t* ids;  // null: one weight
  int n_rows, E;       // E 0: one weight
  int waves;           // of a workgroup
  int by_row;          // a place per row, not per expert
};

// Has the lines of the struct requested together, at the kernel's start.
__device__ __forceinline__ void fetch_args(const W4Args& a) {
  asm volatile("" ::"s"(a.w), "s"(a.x), "s"(a.K), "s"(a.panel), "s"(a.out_vec));
}

// The value as one the compiler cannot trace: what is computed from it stays
// where it is written, not in registers kept from the kernel's start.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The x row of a row.
__device__ __forceinline__ uint32_t x_row(const W4Args& a, uint32_t row) {
  const uint32_t q = __umulhi(row, a.topk_magic);  // or one less
  return row - q * a.topk >= a.topk ? q + 1 : q;
}

// The bits of unpack()'s bytes that a word holds, and the lowest of the magnitude,
// which it does not. The mask in a scalar register and the other in a vector one
// make an and and an or one operation. Taken once, at a kernel's start: the
// statements are opaque to the compiler, which would move a mask it knows across
// the reversal, and could not keep the vector one clear of an MFMA's registers
// further down.
struct Codes {
  uint32_t mask, low;
};
__device__ __forceinline__ Codes codes() {
  Codes c;
  asm volatile("s_mov_b32 %0, 0x8e8e8e8e" : "=s"(c.mask));
  asm volatile("v_mov_b32 %0, 0x01010101" : "=v"(c.low));
  return c;
}

// 8 packed values of one column -> the bf16 values v - 7.5.
__device__ __forceinline__ u32x4 unpack(uint32_t w, Codes c) {
  constexpr float kScale = 256.f;  // of (2 v - 15) / 512
  const int a = (int)((w & c.mask) | c.low);
  const int b = (int)((__builtin_bitreverse32(w) & c.mask) | c.low);
  auto pair = [](auto v) { return __builtin_bit_cast(uint32_t, v); };
  u32x4 r;
  r[0] = pair(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, kScale, false));
  r[1] = pair(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, kScale, true));
  r[2] = pair(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, kScale, false));
  r[3] = pair(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, kScale, true));
  return r;
}

// x operand of one k step as loaded: 8 bf16 or 8 fp32 values.
template <bool F32>
struct XRaw {
  u32x4 v[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ XRaw<F32> load_x(rsrc_t rx, uint32_t row_off, int k, int K) {
  XRaw<F32> f;
  uint32_t off = row_off + (uint32_t)k * (F32 ? 4u : 2u);
  off = row_off != kPast && k < K ? off : kPast;
  f.v[0] = ld16(rx, off);
  if constexpr (F32) f.v[1] = ld16(rx, off + 16u);  // kPast + 16 is past every buffer's end
  return f;
}

// The operand's bf16 parts: the values, or an fp32 value's three parts,
// smallest first.
template <bool F32>
struct XFrag {
  static constexpr int kParts = F32 ? 3 : 1;
  u32x4 p[kParts];
  __device__ __forceinline__ void set(const XRaw<F32>& r) {
    if constexpr (!F32) {
      p[0] = r.v[0];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float v0 = __uint_as_float(r.v[i >> 1][(i & 1) * 2]);
        const float v1 = __uint_as_float(r.v[i >> 1][(i & 1) * 2 + 1]);
        const uint32_t h = pack_bf16(v0, v1);
        const float r0 = v0 - lo_f(h), r1 = v1 - hi_f(h);
        const uint32_t m = pack_bf16(r0, r1);
        p[2][i] = h;
        p[1][i] = m;
        p[0][i] = pack_bf16(r0 - lo_f(m), r1 - hi_f(m));
      }
    }
  }
};

// Where a chunk of one pair of tiles lies. Built from scalars, so that a load
// needs no loop over lanes; a chunk that is not there reads as 0.
struct ChunkAt {
  rsrc_t w, s, z;
  bool whole;

  template <int SG, int ES, bool ZP>
  __device__ __forceinline__ void set(const W4Args& a, const uint8_t* pw, const uint8_t* ps,
                                      const uint8_t* pz, int c, bool in) {
    constexpr uint32_t kCell = 32u * SG;
    whole = c < (a.ksteps >> 2);
    const uint32_t blk = SG > 1 ? (uint32_t)c : __umulhi(2u * (uint32_t)c, a.block_magic);
    w = buf(pw, in ? 2048u : 0u);
    s = buf(ps + (uint64_t)blk * (kCell * ES), in ? kCell * ES : 0u);
    z = s;
    if constexpr (ZP) z = buf(pz + (uint64_t)blk * kCell, in ? kCell : 0u);
  }
};

// The weights of one chunk (128 k values) of NT column tiles of a pair, as
// loaded, and both tiles' scales and zero points.
template <bool F32, int SG, bool ZP, int NT>
struct WChunk {
  static constexpr int kEs = F32 ? 4 : 2;
  static constexpr int kWords = SG * kEs / 2;
  static constexpr int kLoads = NT + (kWords + 3) / 4 + (ZP ? 1 : 0);
  u32x4 w[NT];
  uint32_t s[kWords];
  uint32_t z[ZP ? (SG + 1) / 2 : 1];

  // t0: the pair's first tile to load (0 for both)
  __device__ __forceinline__ void load(const W4Args& a, const ChunkAt& at, int t0, int lane) {
    const uint32_t left = (uint32_t)(a.ksteps & 3);
    // offsets wholly in the vector operand: the range check is against it
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t o = at.whole ? (uint32_t)lane * 16u + (t0 + nt) * 1024u
                                  : (uint32_t)lane * 4u * left + (t0 + nt) * 256u * left;
      w[nt] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(at.w, o, 0, kNT));
    }
    const uint32_t col = (uint32_t)lane & 15u;
    words<kWords>(s, at.s, col * (kWords * 4u));
    if constexpr (ZP && SG == 1)
      z[0] = __builtin_amdgcn_raw_buffer_load_b16(at.z, col * 2u, 0, 0);
    else if constexpr (ZP)
      words<SG / 2>(z, at.z, col * (SG * 2u));
  }
  template <int N>
  static __device__ __forceinline__ void words(uint32_t* d, rsrc_t r, uint32_t off) {
    if constexpr (N == 1) {
      d[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
    } else if constexpr (N == 2) {
      const u32x2 v = __builtin_bit_cast(u32x2,
                                         __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
      d[0] = v[0];
      d[1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const u32x4 v = __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + i * 4u, 0, 0));
        d[i] = v[0];
        d[i + 1] = v[1];
        d[i + 2] = v[2];
        d[i + 3] = v[3];
      }
    }
  }
  // of group sg and tile t of the pair; the zero point with the offset of unpack()
  __device__ __forceinline__ float scale(int sg, int t) const {
    if constexpr (F32)
      return __uint_as_float(t ? s[sg * 2 + 1] : s[sg * 2]);
    else
      return t ? hi_f(s[sg]) : lo_f(s[sg]);
  }
  __device__ __forceinline__ float zero(int sg, int t) const {
    return (float)((z[sg / 2] >> (16 * (sg & 1) + 8 * t)) & 0xffu) - 7.5f;
  }
};

// Minus the sum of x that a group's sums start from, times 0.5 (8 - 7.5) where
// every zero point is 8: bf16 pairs of -1 and -0.5.
constexpr uint32_t minus_ones(bool zp) { return zp ? 0xbf80bf80u : 0xbf00bf00u; }

// acc += the chunk's products, group by group. `x(mb, ks, f)` fills f with the
// bf16 parts of k step ks of row block mb. `sum(mb, sg)`, if given, is minus the
// sum of that group's x; else MFMAs with a constant operand take it.
struct NoSums {};
template <bool F32, int SG, bool ZP, int NT, int MB, typename X, typename S = NoSums>
__device__ __forceinline__ void add_chunk(const WChunk<F32, SG, ZP, NT>& wc, int t0, X x,
                                          Codes cd, f32x4 (&acc)[NT][MB], S sum = S{}) {
  constexpr bool kSums = !std::is_same<S, NoSums>::value;
  constexpr int kPer = 4 / SG, kParts = XFrag<F32>::kParts;
  constexpr uint32_t kc = minus_ones(ZP);
  const u32x4 cons = {kc, kc, kc, kc};
#pragma unroll
  for (int sg = 0; sg < SG; ++sg) {
    XFrag<F32> f[MB][kPer];
    f32x4 dc[MB] = {};
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      if constexpr (kSums) dc[mb] = sum(mb, sg);
#pragma unroll
      for (int ks = 0; ks < kPer; ++ks) x(mb, sg * kPer + ks, f[mb][ks]);
    }
    if constexpr (!kSums) {
#pragma unroll
      for (int ks = 0; ks < kPer; ++ks)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int p = 0; p < kParts; ++p) dc[mb] = mfma(f[mb][ks].p[p], cons, dc[mb]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 t[MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        t[mb] = dc[mb];
        if constexpr (ZP) {
          const float z = wc.zero(sg, t0 + nt);
#pragma unroll
          for (int i = 0; i < 4; ++i) t[mb][i] *= z;
        }
      }
#pragma unroll
      for (int ks = 0; ks < kPer; ++ks) {
        const u32x4 wf = unpack(wc.w[nt][sg * kPer + ks], cd);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int p = 0; p < kParts; ++p) t[mb] = mfma(f[mb][ks].p[p], wf, t[mb]);
      }
      const float sc = wc.scale(sg, t0 + nt);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][mb][i] = fmaf(sc, t[mb][i], acc[nt][mb][i]);
    }
    // operands of the next chunk (fp32, with three parts, and small groups: of the
    // next group) are not fetched into registers ahead, which the weights in flight
    // need
    if (F32 || SG == 4 || sg == SG - 1) __builtin_amdgcn_sched_barrier(0);
  }
}

template <typename Row>
__device__ __forceinline__ void store4(typename Row::elem* o, f32x4 v, int left, bool vec) {
  if (vec && left >= 4) {
    if constexpr (sizeof(typename Row::elem) == 4)
      *reinterpret_cast<f32x4*>(o) = v;
    else
      *reinterpret_cast<u32x2*>(o) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) o[j] = Row::narrow(v[j]);
  }
}

// 16 bytes of each lane straight into LDS, lane l's at p + l.
__device__ __forceinline__ void load_to_lds(rsrc_t r, u32x4* p, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      r, (__attribute__((address_space(3))) void*)p, 16, off, 0, 0, 0);
}
// Waits until at most N of the wave's loads are outstanding (the last requested
// ones: loads return in order).
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "the counter has 6 bits");
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  // vmcnt in bits 3:0 and 15:14; expcnt and lgkmcnt left at their maxima
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0f70);
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Workgroup barrier that orders LDS only: requested weights stay in flight
// across it (no kernel here passes global memory between its waves).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A workgroup's place, blockIdx.y, is an expert; in calls of fewer rows than
// experts (by_row) it is a row, and stands for that row's expert where no
// earlier row has the same. Returns the expert, -1 for none.
__device__ __forceinline__ int place_expert(const W4Lead& l) {
  const int y = (int)blockIdx.y;
  const int e = l.E > 0 && l.by_row ? uniform_i32(l.ids[y]) : y;
  return l.E > 0 && (uint32_t)e >= (uint32_t)l.E ? -1 : e;
}

// A segment's ids, in runs of 64 * rounds per wave, four rounds at a time. The
// first four are requested ahead of a workgroup's weights.
struct IdRun {
  rsrc_t r;
  int rounds, first;
  int id[4];

  __device__ __forceinline__ void set(const W4Lead& l, int seg, int len, int wave, int lane) {
    rounds = (len + 64 * l.waves - 1) / (64 * l.waves);  // <= 32
    first = wave * rounds * 64 + lane;
    r = buf(l.ids + seg, l.E > 0 ? (uint32_t)len * 4u : 0u);  // past the end: 0
    load(0);
  }
  __device__ __forceinline__ void load(int r0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      id[i] = (int)__builtin_amdgcn_raw_buffer_load_b32(r, (first + (r0 + i) * 64) * 4, 0, 0);
  }
};

// The rows of [seg, seg + len) of one workgroup: those whose id is its expert e
// from the front of `list` (none if an earlier place has them), and from its
// end the rows without an expert that fall to this place (the place's own row,
// or spread over the experts; the workgroup writes their zeros), each in row
// order. Every wave scans a run of 64 * rounds ids and lists its hits behind
// those of the waves before it, so that workgroups which share an expert's rows
// agree on the list.
struct RowList {
  int live, dead;
};

__device__ __forceinline__ int lanes_before(uint64_t m) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32),
                                        __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

__device__ __forceinline__ RowList list_rows(const W4Lead& l, IdRun& run, int e, int seg, int len,
                                             int wave, int* list, int* counts) {
  const int lane = here(threadIdx.x & 63);
  const int E = l.E, rounds = run.rounds, first = run.first;
  const int(&id)[4] = run.id;
  const int y = (int)blockIdx.y;
  const int shift = 32 - __builtin_clz((unsigned)len);       // len < 2^shift
  uint32_t hits = 0, drops = 0;
  int n_hits = 0, n_drops = 0;
  for (int r0 = 0; r0 < rounds; r0 += 4) {
    if (r0 > 0) run.load(r0);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = first + (r0 + r) * 64;
      const bool in = r0 + r < rounds && i < len;
      const bool hit = in && id[r] == e && e >= 0;
      const int owner = l.by_row ? i : (int)(((uint32_t)i * (uint32_t)E) >> shift);
      const bool drop = in && (uint32_t)id[r] >= (uint32_t)E && owner == y;
      n_hits += __popcll(__ballot(hit));
      n_drops += __popcll(__ballot(drop));
      hits |= (hit ? 1u : 0u) << ((r0 + r) & 31);
      drops |= (drop ? 1u : 0u) << ((r0 + r) & 31);
    }
  }
  if (seg > 0) lds_barrier();  // the list's last readers are done
  if (lane == 0) counts[wave] = n_hits | n_drops << 16;
  lds_barrier();
  int at = 0, all = 0;
  static_assert(kMaxWaves % 4 == 0, "counts are read four at a time");
#pragma unroll
  for (int w = 0; w < kMaxWaves; w += 4) {
    const i32x4 c = *reinterpret_cast<const i32x4*>(counts + w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      at += w + i < wave ? c[i] : 0;
      all += w + i < l.waves ? c[i] : 0;
    }
  }
  at = uniform_i32(at);
  all = uniform_i32(all);
  int at_hit = at & 0xffff, at_drop = at >> 16;
  if ((n_hits | n_drops) > 0) {
    for (int r = 0; r < rounds; ++r) {
      const bool hit = (hits >> r) & 1, drop = (drops >> r) & 1;
      const uint64_t mh = __ballot(hit), md = __ballot(drop);
      if (hit) list[at_hit + lanes_before(mh)] = seg + first + r * 64;
      if (drop) list[kScan - 1 - at_drop - lanes_before(md)] = seg + first + r * 64;
      at_hit += __popcll(mh);
      at_drop += __popcll(md);
    }
  }
  lds_barrier();
  int live = all & 0xffff;
  if (l.by_row && live > 0 && uniform_i32(list[0]) != y) live = 0;
  return RowList{live, all >> 16};
}

// Zeros into columns [n0, n0 + cols) of the rows listed from the end, a wave per
// row.
template <typename Row>
__device__ __forceinline__ void zero_rows(const W4Args& a, const int* list, int dead, int n0,
                                          int cols, int wave, int waves) {
  const int lane = here(threadIdx.x & 63);
  const int n1 = min(n0 + cols, a.N);
  for (int r = wave; r < dead; r += waves) {
    typename Row::elem* o = static_cast<typename Row::elem*>(a.out) +
                            (int64_t)uniform_i32(list[kScan - 1 - r]) * a.out_ld;
    for (int n = n0 + lane * 4; n < n1; n += 256)
      store4<Row>(o + n, f32x4{0.f, 0.f, 0.f, 0.f}, n1 - n, a.out_vec != 0);
  }
}

// Few column tiles: a workgroup owns NT tiles, its waves split k and add their
// sums up through LDS in wave order; x goes straight to the operands.
template <bool F32, int SG, bool ZP, int MB, int NT>
__global__ void __launch_bounds__(64 * kSplitWaves)
w4_split_kernel(const int32_t* ids, int n_rows, int E, int waves, int by_row, W4Args a) {
  typedef typename std::conditional<F32, F32Row, Bf16Row>::type Row;
  constexpr int kCols = 16 * NT, kStride = kCols + 4, kRows = 16 * MB;
  __shared__ int list[kScan];
  __shared__ __attribute__((aligned(16))) int counts[kMaxWaves];
  __shared__ float red[kSplitWaves * kRows * kStride];
  const W4Lead lead = {ids, n_rows, E, waves, by_row};
  const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, lg = lane >> 4;
  const int wave = uniform_i32(tid >> 6);
  IdRun run;
  run.set(lead, 0, min(kScan, n_rows), wave, lane);
  fetch_args(a);
  const Codes cd = codes();
  const int e = place_expert(lead), tile = (int)blockIdx.x * NT;
  const int n0 = tile * 16, chunks = (a.ksteps + 3) >> 2;
  typename Row::elem* out = static_cast<typename Row::elem*>(a.out);
  const rsrc_t rx = buf(a.x, a.x_bytes);
  constexpr int kCell = 32 * SG;
  const int64_t ep = (int64_t)max(e, 0) * a.pairs + (tile >> 1);
  const uint8_t* pw = a.w + ep * a.ksteps * 512;
  const uint8_t* ps = a.s + ep * a.blocks * (kCell * (F32 ? 4 : 2));
  const uint8_t* pz = a.z + (ZP ? ep * a.blocks * kCell : 0);
  const int t0 = NT == 1 ? tile & 1 : 0;
  WChunk<F32, SG, ZP, NT> wc;
  auto request = [&](int c) {
    ChunkAt at;
    at.set<SG, (F32 ? 4 : 2), ZP>(a, pw + (int64_t)c * 2048, ps, pz, c, c < chunks);
    wc.load(a, at, t0, lane);
  };
  request(wave);  // the first chunk's weights, ahead of the rows they meet
  bool primed = true;

  for (int seg = 0; seg < n_rows; seg += kScan) {
    const int len = min(kScan, n_rows - seg);
    int n_list = len;
    if (E > 0) {
      if (seg > 0) run.set(lead, seg, len, wave, lane);
      const RowList l = list_rows(lead, run, e, seg, len, wave, list, counts);
      n_list = l.live;
      if (l.dead > 0 && blockIdx.z == 0)
        zero_rows<Row>(a, list, l.dead, n0, kCols, wave, waves);
    }
    for (int b0 = (int)blockIdx.z * kRows; b0 < n_list; b0 += (int)gridDim.z * kRows) {
      uint32_t row_off[MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const int at = b0 + mb * 16 + li;
        const int row = at < n_list ? (E > 0 ? list[at] : seg + at) : -1;
        row_off[mb] = row >= 0 ? x_row(a, (uint32_t)row) * a.x_ld_bytes : kPast;
      }
      if (!primed) request(wave);
      primed = false;
      f32x4 acc[NT][MB] = {};
      for (int c = wave; c < chunks; c += waves) {
        XRaw<F32> x[MB][4];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            x[mb][ks] = load_x<F32>(rx, row_off[mb], c * 128 + ks * 32 + lg * 8, a.K);
        // bf16: all of them requested ahead of the first product's wait, which the
        // compiler else puts between them; fp32 rows, whose conversions it spreads
        // over the loads, take 8.0 us without and 8.3 with (5 of 1000 x 1365, 37 rows)
        if constexpr (!F32) __builtin_amdgcn_sched_barrier(0);
        add_chunk<F32, SG, ZP, NT, MB>(
            wc, t0, [&](int mb, int ks, XFrag<F32>& f) { f.set(x[mb][ks]); }, cd, acc);
        if (c + waves < chunks) request(c + waves);
      }
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            red[(wave * kRows + mb * 16 + lg * 4 + i) * kStride + nt * 16 + li] = acc[nt][mb][i];
      lds_barrier();
      for (int i = tid; i < kRows * (kCols / 4); i += 64 * waves) {
        const int r = i / (kCols / 4), c4 = i % (kCols / 4) * 4;
        f32x4 sum = *reinterpret_cast<const f32x4*>(&red[r * kStride + c4]);
        for (int w = 1; w < waves; ++w)
          sum += *reinterpret_cast<const f32x4*>(&red[(w * kRows + r) * kStride + c4]);
        if (b0 + r >= n_list) continue;
        const int64_t row = E > 0 ? list[b0 + r] : seg + b0 + r;
        store4<Row>(out + row * a.out_ld + n0 + c4, sum, a.N - n0 - c4, a.out_vec != 0);
      }
      lds_barrier();
    }
  }
}

// Many column tiles: x rows go into LDS once per workgroup, as the operands the
// MFMAs take (k in panels where the rows do not fit whole);
// each wave then streams whole columns: pairs of tiles over all of k, kAhead
// chunks of weights requested ahead, no barrier between.
template <bool F32, int SG, bool ZP, int MB>
__global__ void __launch_bounds__(64 * kMaxWaves, simd_waves(F32, MB))
w4_stream_kernel(const int32_t* ids, int n_rows, int E, int waves, int by_row, int k_waves,
                 W4Args a) {
  typedef typename std::conditional<F32, F32Row, Bf16Row>::type Row;
  typedef WChunk<F32, SG, ZP, kPair> Chunk;
  constexpr int kRows = 16 * MB, kParts = XFrag<F32>::kParts;
  __shared__ int list[kScan];
  __shared__ __attribute__((aligned(16))) int counts[kMaxWaves];
  extern __shared__ u32x4 xs[];  // [k step][row block][part][lane]
  const W4Lead lead = {ids, n_rows, E, waves, by_row};
  const int tid = threadIdx.x, lane = tid & 63, li = lane & 15, lg = lane >> 4;
  const int wave = uniform_i32(tid >> 6);
  IdRun run;
  run.set(lead, 0, min(kScan, n_rows), wave, lane);
  fetch_args(a);
  const int panel = a.panel;
  // behind the operands, minus the sums of x: [group][row block][row]
  f32x4* x_sums = reinterpret_cast<f32x4*>(xs + panel * (4 * MB * kParts * 64));
  const Codes cd = codes();
  const int e = place_expert(lead), slice = (int)blockIdx.x;
  const int chunks = (a.ksteps + 3) >> 2;
  typename Row::elem* out = static_cast<typename Row::elem*>(a.out);
  const rsrc_t rx = buf(a.x, a.x_bytes);
  // kw waves share a pair, each every kw-th chunk; a wave's pairs: every wn-th
  // of the slice's
  const int kw = k_waves, n_wn = a.pair_waves;
  const int wn = kw == 1 ? wave : kw == 2 ? wave >> 1 : kw == 4 ? wave >> 2 : wave * 11 >> 5;
  const int wk = wave - wn * kw;  // kw <= 4, and wave * 11 / 32 = wave / 3 up to 15
  const int pair0 = slice * a.per_slice + wn;
  const int left = max(0, min((slice + 1) * a.per_slice, a.pairs) - pair0) + n_wn - 1;
  const int all_pairs = n_wn == 1 ? left : (int)__umulhi((uint32_t)left, a.wave_magic);
  const int n_pairs = uniform_i32(e < 0 ? 0 : all_pairs);
  // A pair takes whole turns of the ring: places past its chunks stay empty.
  const int turns = a.turns;
  constexpr int kEs = F32 ? 4 : 2, kCell = 32 * SG;
  const int64_t ep = (int64_t)max(e, 0) * a.pairs + pair0;
  const int64_t w_pair = (int64_t)a.ksteps * 512, s_pair = (int64_t)a.blocks * kCell;
  const uint8_t* const pw0 = a.w + ep * w_pair;
  const uint8_t* const ps0 = a.s + ep * s_pair * kEs;
  const uint8_t* const pz0 = a.z + (ZP ? ep * s_pair : 0);
  int lp, lj, lc;  // pair, turn place and chunk of the next request
  const uint8_t *pw, *ps, *pz;
  auto first_request = [&] {
    lp = lj = 0;
    lc = wk;
    pw = pw0;
    ps = ps0;
    pz = pz0;
  };
  auto request = [&](Chunk& w) {
    ChunkAt at;
    at.set<SG, kEs, ZP>(a, pw + (int64_t)lc * 2048, ps, pz, lc, lp < n_pairs && lc < chunks);
    w.load(a, at, 0, lane);
    // requests stay in order, so that a wait for one leaves the later ones out
    __builtin_amdgcn_sched_barrier(0);
    lc += kw;
    if (++lj == turns) {
      lj = 0;
      lc = wk;
      ++lp;
      pw += n_wn * w_pair;
      ps += n_wn * s_pair * kEs;
      pz += ZP ? n_wn * s_pair : 0;
    }
  };

  // The first weights are requested ahead of the rows they meet, the others once x
  // has been, so that weights arrive while x does (128 experts of 2048 x 768, 640
  // rows: 23.4 us, all of them after x 24.2).
  constexpr int kEarly = 1;
  Chunk ring[kAhead];
  auto first_requests = [&] {
    first_request();
#pragma unroll
    for (int d = 0; d < kEarly; ++d) request(ring[d]);
  };
  first_requests();
  bool primed = true;

  for (int seg = 0; seg < n_rows; seg += kScan) {
    int n_list = min(kScan, n_rows - seg);
    if (E > 0) {
      if (seg > 0) run.set(lead, seg, n_list, wave, lane);
      const RowList l = list_rows(lead, run, e, seg, n_list, wave, list, counts);
      n_list = l.live;
      if (l.dead > 0 && blockIdx.z == 0)
        zero_rows<Row>(a, list, l.dead, slice * a.per_slice * kPair * 16,
                       a.per_slice * kPair * 16, wave, waves);
    }
    const int step = (int)gridDim.z * kRows;
    for (int b0 = (int)blockIdx.z * kRows; b0 < n_list; b0 += step) {
      uint32_t row_off[MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const int at = b0 + mb * 16 + here(li);
        const int row = at < n_list ? (E > 0 ? list[at] : seg + at) : -1;
        row_off[mb] = row >= 0 ? x_row(a, (uint32_t)row) * a.x_ld_bytes : kPast;
      }
      // the sums of a pair's tile and row block into the rows of out
      auto store = [&](int pair, int nt, int mb, f32x4 v) {
        const int l = here(tid & 63), n = pair * (kPair * 16) + nt * 16 + (l & 15);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = b0 + mb * 16 + (l >> 4) * 4 + i;
          if (at >= n_list || n >= a.N) continue;
          const int row = E > 0 ? list[at] : seg + at;
          out[(int64_t)row * a.out_ld + n] = Row::narrow(v[i]);
        }
      };
      // x into LDS, k step by k step, the waves in turn. bf16 operands go there
      // directly, all in flight; fp32 rows pass through registers on their way
      // into parts.
      auto stage = [&](int p0, int steps) {
        const int lane = here(tid & 63), lg = lane >> 4;
        if constexpr (!F32) {
          for (int f = wave; f < steps; f += waves) {
            const int k = p0 * 128 + f * 32 + lg * 8;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
              load_to_lds(rx, xs + (f * MB + mb) * 64,
                          row_off[mb] != kPast && k < a.K ? row_off[mb] + k * 2u : kPast);
          }
        } else {
          constexpr int kBatch = 4;
          for (int f0 = wave; f0 < steps; f0 += kBatch * waves) {
            XRaw<F32> r[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int f = f0 + i * waves;
              r[i] = load_x<F32>(rx, row_off[0], f < steps ? p0 * 128 + f * 32 + lg * 8 : a.K, a.K);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int f = f0 + i * waves;
              if (f < steps) {
                XFrag<F32> q;
                q.set(r[i]);
#pragma unroll
                for (int p = 0; p < kParts; ++p) xs[(f * kParts + p) * 64 + lane] = q.p[p];
              }
            }
          }
        }
      };
      // The operands of a last k step past K hold zeros whatever a load past a
      // buffer's end leaves in LDS.
      auto stage_end = [&](int p0, int p1) {
        const int lane = here(tid & 63), lg = lane >> 4;
        if constexpr (!F32) {
          if (p1 * 128 > a.K) {
            for (int f = wave; f < (p1 - p0) * 4; f += waves) {
              if (p0 * 128 + f * 32 + lg * 8 < a.K) continue;
#pragma unroll
              for (int mb = 0; mb < MB; ++mb) xs[(f * MB + mb) * 64 + lane] = u32x4{0, 0, 0, 0};
            }
          }
        }
      };
      // The groups' sums of x, the waves in turn.
      auto sum_groups = [&](int groups) {
        constexpr int kPer = 4 / SG;
        constexpr uint32_t kc = minus_ones(ZP);
        const u32x4 cons = {kc, kc, kc, kc};
        const int lane = here(tid & 63), li = lane & 15, lg = lane >> 4;
#pragma unroll 1
        for (int g = wave; g < groups; g += waves) {
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < kPer; ++ks)
#pragma unroll
              for (int p = 0; p < kParts; ++p)
                d = mfma(xs[(((g * kPer + ks) * MB + mb) * kParts + p) * 64 + lane], cons, d);
            if (li == 0) x_sums[(g * MB + mb) * 4 + lg] = d;
          }
        }
      };
      f32x4 acc[kPair][MB];
      if (!primed) first_requests();
      primed = false;
      lds_barrier();  // the last block's readers are done
      stage(0, min(panel, chunks) * 4);
      // x's loads stay ahead of these requests, which the wait below counts
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = kEarly; d < kAhead; ++d) request(ring[d]);
      for (int p0 = 0, j0 = 0; p0 < chunks; p0 += panel, j0 += a.panel_turns) {
        const int p1 = min(p0 + panel, chunks);
        if (p0 > 0) {
          lds_barrier();
          stage(p0, (p1 - p0) * 4);
        }
        if constexpr (!F32) {
          if (p0 > 0)
            wait_loads<0>();
          else
            wait_loads<Chunk::kLoads *(kAhead - kEarly)>();
        }
        stage_end(p0, p1);
        lds_barrier();
        sum_groups((p1 - p0) * SG);
        lds_barrier();
        // one panel: every pair; several, or several waves a pair: the one pair's
        // share of them
        for (int pair = 0; pair < n_pairs; ++pair) {
          if (p0 == 0) {
#pragma unroll
            for (int nt = 0; nt < kPair; ++nt)
#pragma unroll
              for (int mb = 0; mb < MB; ++mb) acc[nt][mb] = f32x4{0.f, 0.f, 0.f, 0.f};
          }
          for (int c0 = wk + j0 * kw; c0 < p1; c0 += kAhead * kw) {
#pragma unroll
            for (int d = 0; d < kAhead; ++d) {
              const int c = c0 + d * kw;
              if (c < p1) {
                const u32x4* px = xs + (c - p0) * (4 * MB * kParts * 64) + lane;
                auto operand = [&](int mb, int ks, XFrag<F32>& f) {
#pragma unroll
                  for (int p = 0; p < kParts; ++p) f.p[p] = px[((ks * MB + mb) * kParts + p) * 64];
                };
                const f32x4* px_sums = x_sums + (c - p0) * (SG * MB * 4) + lg;
                add_chunk<F32, SG, ZP, kPair, MB>(
                    ring[d], 0, operand, cd, acc,
                    [&](int mb, int sg) { return px_sums[(sg * MB + mb) * 4]; });
              }
              request(ring[d]);
            }
          }
          if (p1 < chunks || kw > 1) continue;
#pragma unroll
          for (int nt = 0; nt < kPair; ++nt)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) store(pair0 + pair * n_wn, nt, mb, acc[nt][mb]);
        }
      }
      if (kw == 1) continue;
      // the sums of a pair's waves, added in wave order, in the LDS of x
      lds_barrier();
      f32x4* red = reinterpret_cast<f32x4*>(xs) + here(lane);  // [wave][tile][row block][lane]
      if (n_pairs > 0) {
#pragma unroll
        for (int nt = 0; nt < kPair; ++nt)
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
            red[((wave * kPair + nt) * MB + mb) * 64] = acc[nt][mb];
      }
      lds_barrier();
#pragma unroll
      for (int nt = 0; nt < kPair; ++nt) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          if (n_pairs == 0 || (nt * MB + mb) % kw != wk) continue;
          f32x4 sum = {0.f, 0.f, 0.f, 0.f};
          for (int w = 0; w < kw; ++w)
            sum += red[(((wn * kw + w) * kPair + nt) * MB + mb) * 64];
          store(pair0, nt, mb, sum);
        }
      }
    }
  }
}

template <bool F32, int SG, bool ZP, int MB>
void launch_w4(const W4Args& a0, const W4Plan& p, W4Rows rows, hipStream_t s) {
  W4Args a = a0;
  const int32_t* ids = rows.ids;
  const int n_rows = rows.n, E = rows.ids ? rows.experts : 0;
  a.per_slice = p.per_slice;
  a.pair_waves = p.waves / p.k_waves;
  a.wave_magic = (uint32_t)(((1ull << 32) + a.pair_waves - 1) / a.pair_waves);
  const dim3 grid((unsigned)p.slices, (unsigned)p.places, (unsigned)p.splits), block(64 * p.waves);
  if (!p.stream) {
    // two tiles: calls of several passes, which have two row blocks or fp32 rows
    if constexpr (F32 || MB > 1) {
      if (p.tiles == 2) {
        hipLaunchKernelGGL((w4_split_kernel<F32, SG, ZP, MB, 2>), grid, block, 0, s, ids, n_rows,
                           E, p.waves, (int)p.by_row, a);
        return;
      }
    }
    hipLaunchKernelGGL((w4_split_kernel<F32, SG, ZP, MB, 1>), grid, block, 0, s, ids, n_rows, E,
                       p.waves, (int)p.by_row, a);
    return;
  }
  const int chunks = (a.ksteps + 3) / 4, turn = kAhead * p.k_waves;
  a.panel = panel_chunks(F32, MB, SG) / turn * turn;
  if (chunks <= panel_chunks(F32, MB, SG)) a.panel = chunks;
  a.panel_turns = a.panel / p.k_waves;
  a.turns = ((chunks + p.k_waves - 1) / p.k_waves + kAhead - 1) / kAhead * kAhead;
  size_t lds = (size_t)a.panel * chunk_lds(F32, MB, SG);
  const size_t sums = (size_t)p.waves * kPair * MB * 1024;
  if (p.k_waves > 1 && lds < sums) lds = sums;
  hipLaunchKernelGGL((w4_stream_kernel<F32, SG, ZP, MB>), grid, block, lds, s, ids, n_rows, E,
                     p.waves, (int)p.by_row, p.k_waves, a);
}

template <int SG, bool ZP>
void dispatch_w4_sg(const W4Args& a, const W4Plan& p, bool f32, W4Rows rows, hipStream_t s) {
  if (f32) return launch_w4<true, SG, ZP, 1>(a, p, rows, s);
  if (p.mb == 2) return launch_w4<false, SG, ZP, 2>(a, p, rows, s);
  launch_w4<false, SG, ZP, 1>(a, p, rows, s);
}

void dispatch_w4(const W4Args& a, const W4Plan& p, bool f32, int sg, W4Rows rows,
                 hipStream_t s) {
  if (a.z) {
    if (sg == 4) return dispatch_w4_sg<4, true>(a, p, f32, rows, s);
    if (sg == 2) return dispatch_w4_sg<2, true>(a, p, f32, rows, s);
    return dispatch_w4_sg<1, true>(a, p, f32, rows, s);
  }
  if (sg == 4) return dispatch_w4_sg<4, false>(a, p, f32, rows, s);
  if (sg == 2) return dispatch_w4_sg<2, false>(a, p, f32, rows, s);
  dispatch_w4_sg<1, false>(a, p, f32, rows, s);
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
  a.cells = (int64_t)n_experts * l.pairs * l.blocks * 32 * l.sg;
  a.K = k_in;
  a.N = n_out;
  a.group = group;
  a.groups = (int32_t)(((int64_t)k_in + group - 1) / group);  // group may be near 2^31
  a.pairs = (int32_t)l.pairs;
  a.ksteps = (int32_t)l.ksteps;
  a.blocks = (int32_t)l.blocks;
  a.sg = (int32_t)l.sg;
  const int64_t groups = (a.words + a.cells + 255) / 256;
  if (groups > kMaxRows) return fail(MLORA_ERR_INVALID, "%s: weights too large", who);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (dtype == MLORA_BF16)
    hipLaunchKernelGGL(w4_pack_kernel<Bf16Row>, flat_grid(groups), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(w4_pack_kernel<F32Row>, flat_grid(groups), dim3(256), 0, s, a);
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
  a.out_ld = out_ld;
  a.x_bytes = (uint32_t)(((need - 1) * x_ld + route->k_in) * es);
  a.x_ld_bytes = (uint32_t)(x_ld * es);
  a.topk = x_by_row ? 1u : (uint32_t)top_k;
  a.topk_magic = 0xffffffffu / a.topk;
  a.K = route->k_in;
  a.N = route->n_out;
  a.pairs = (int32_t)l.pairs;
  a.ksteps = (int32_t)l.ksteps;
  a.blocks = (int32_t)l.blocks;
  const uint32_t per_block = route->group <= 128 ? 1u : (uint32_t)route->group / 128u;
  a.block_magic = ((1u << 31) + per_block - 1) / per_block;
  a.out_vec = out_ld % 4 == 0 && aligned(out, 4 * es);
  const bool f32 = route->dtype == MLORA_F32;
  (void)hipGetLastError();
  const W4Rows rows = {ids, (int32_t)n_rows, route->n_experts};
  const W4Plan p = plan_w4(route, rows, f32, (int)l.sg);
  dispatch_w4(a, p, f32, (int)l.sg, rows, reinterpret_cast<hipStream_t>(stream));
  return launch_status(who);
}
