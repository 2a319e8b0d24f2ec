// A whole MoE layer for a few tokens in two kernels, for gfx950 (MI355X): the
// router's choice, gate and up with their activation; down and the weighted sum.
#include "mlora_fp8.h"
#include "mlora_router.h"

namespace mlora {
namespace {

// out[t] = sum over j of p[t, j] down_e (silu(gate_e x[t]) * (up_e x[t])), e the
// j-th expert of token t. The weights of the chosen experts are read once, as
// E4M3 codes that become bf16 values (exactly) in front of bf16 MFMAs of 16
// weight rows by 16 tokens; every token of the call is a column of them, and the
// ones that did not choose the expert are left out of the result. x stays as it
// is: a bf16 value is one operand, an fp32 value three (24 bits). The activated
// rows, times p, pass from kernel to kernel in fp32 and become three operands there. A
// block's sums enter the fp32 sums times its scale.
//
// Kernel one: each workgroup chooses every token's experts itself (the logits
// are a few KB), lists the experts that are chosen, and takes tiles of 16 hidden
// columns of them in turn; its waves share the blocks of k. Kernel two: a
// workgroup owns 32 out columns and its waves share the experts' blocks, so that
// the sum over the experts needs no atomics. Which wave takes a block goes by the
// expert and the block alone: a token's sums have the same order, and its row the
// same bits, whatever the other tokens choose.

constexpr int kTokens = 16;
constexpr int kWaves = 8;
constexpr int kNone = 255;

struct LayerArgs {
  const void* logits;
  int64_t logits_ld;
  const void* x;
  int64_t x_ld;
  const uint8_t *gate, *up, *down;
  const float *gate_s, *up_s, *down_s;
  void* out;
  int64_t out_ld;
  int32_t* indices;  // may be null
  float* weights;    // may be null
  int32_t* head;     // workspace: count, experts [max_active], slots [max_active][16]
  int32_t* count;    // workspace: splits that are done, of each tile of out
  float* sums;       // workspace: [tiles of out][splits][4][64]
  float* act;        // workspace: [T * k][hidden, whole blocks]
  uint32_t act_bytes;
  int32_t T, E, k, renorm, dim, hidden, DB, HB, max_active;
};

template <typename Row>
constexpr int parts_of_x() { return sizeof(typename Row::elem) == 2 ? 1 : 3; }

// f as P bf16 values whose sum it is, the largest first.
template <int P>
__device__ __forceinline__ void split8(const float* f, u32x4 (&out)[P]) {
  float left[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) left[i] = f[i];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    out[p] = Bf16Row::narrow16(left);
    if (p + 1 < P) {
      float part[8];
      Bf16Row::widen16(out[p], part);
#pragma unroll
      for (int i = 0; i < 8; ++i) left[i] -= part[i];
    }
  }
}

// A block's sums: the tile's 128 products a result, for one or more parts of x.
// Lane group g = lane / 16 holds k = 32 g + 8 j .. + 7 of both operands in step j.
template <int P>
__device__ __forceinline__ f32x4 block_sum(const Fp8Frag& w, const u32x4 (&x)[4][P]) {
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x4 wf = widen_codes(w.h[j / 2][2 * (j % 2)], w.h[j / 2][2 * (j % 2) + 1]);
#pragma unroll
    for (int p = P - 1; p >= 0; --p) s = mfma_bf16(wf, x[j][p], s);
  }
  return s;
}

// Dynamic LDS of kernel one, in words from the start.
struct Lds {
  int ids, wts, flag, place, list, slots, part, total;
};
__host__ __device__ inline Lds lds_of(int n, int E, int max_active) {
  Lds l{};
  l.ids = 0;
  l.wts = l.ids + n;
  l.flag = l.wts + n;
  l.place = l.flag + E;
  l.list = l.place + E;
  l.slots = l.list + max_active;
  l.part = (l.slots + max_active * (kTokens / 4) + 3) & ~3;
  l.total = l.part + 2 * kWaves * 2 * 256;
  return l;
}

// Every token's choice into LDS, by all waves, and a flag for each chosen expert.
// `request` asks for what is needed afterwards, behind the first logits.
template <typename Row, int LPT, int VPL, typename Request>
__device__ __forceinline__ void choose_all(const LayerArgs& a, int* ids, float* wts, int* flag,
                                           bool publish, Request request) {
  const int gl = threadIdx.x & (LPT - 1);
  constexpr int kPer = kWaves * 64 / LPT;
  for (int t0 = 0; t0 < a.T; t0 += kPer) {
    const int t = t0 + (int)(threadIdx.x / LPT);
    float v[VPL];
    load_row<Row, LPT, VPL, Row::kPer16, false>(a.logits, (int64_t)(t < a.T ? t : 0) * a.logits_ld,
                                                a.E, gl, v);
    if (t0 == 0) request();
    int e;
    const float w = choose_experts<Row, LPT, VPL, Row::kPer16>(v, a.E, a.k, a.renorm, gl, &e);
    if (t < a.T && gl < a.k) {
      ids[t * a.k + gl] = e;
      wts[t * a.k + gl] = w;
      flag[e] = 1;
      if (publish && a.indices) a.indices[t * a.k + gl] = e;
      if (publish && a.weights) a.weights[t * a.k + gl] = w;
    }
  }
}

// XB: blocks of k a wave has at most, whose x it keeps in registers; 0: more, and x
// is read again for each tile. SHARE waves share a tile's blocks, and a workgroup takes
// 8 / SHARE neighbouring tiles at a time: with fewer blocks than waves the others had
// nothing to do (16 tokens, top 6 of 68, 154 -> 1153: the layer 34 -> 27 us).
template <typename Row, int XB, int SHARE>
__global__ void __launch_bounds__(64 * kWaves) layer_gate_up_kernel(LayerArgs a) {
  extern __shared__ int lds[];
  constexpr int P = parts_of_x<Row>();
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform_i32(tid >> 6);
  const int n = a.T * a.k;
  const Lds l = lds_of(n, a.E, a.max_active);
  int *ids = lds + l.ids, *place = lds + l.place, *list = lds + l.list;
  float *wts = reinterpret_cast<float*>(lds + l.wts), *part = reinterpret_cast<float*>(lds + l.part);
  uint8_t* slots = reinterpret_cast<uint8_t*>(lds + l.slots);
  const bool first = blockIdx.x == 0;
  int* flag = lds + l.flag;
  for (int e = tid; e < a.E; e += 64 * kWaves) flag[e] = 0;
  for (int i = tid; i < a.max_active * (kTokens / 4); i += 64 * kWaves)
    lds[l.slots + i] = -1;  // four times kNone
  __syncthreads();

  const int t_col = lane & 15, g = lane >> 4;
  const int64_t x_off = (int64_t)min(t_col, a.T - 1) * a.x_ld;
  constexpr int kTiles = kWaves / SHARE;
  const int sub = wave / SHARE, kp = wave % SHARE;
  const int k0 = a.DB * kp / SHARE, k1 = a.DB * (kp + 1) / SHARE;
  typedef Eights<Row, 4> RawX;
  const void* x = static_cast<const typename Row::elem*>(a.x) + x_off;
  auto columns = [&](int kb, int (&k)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = kb * 128 + g * 32 + j * 8;
  };
  auto request_x = [&](int kb, RawX& raw) {
    int k[4];
    columns(kb, k);
    raw.request(x, k, a.dim);
  };
  auto take_x = [&](int kb, RawX& raw, u32x4 (&xf)[4][P]) {
    if (a.dim % 128 != 0) {
      int k[4];
      columns(kb, k);
      raw.finish(k, a.dim);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (P == 1) {
        xf[j][0] = raw.v[j][0];
      } else {
        float v[8];
        raw.widen(j, v);
        split8<P>(v, xf[j]);
      }
    }
  };
  RawX raw[XB > 0 ? XB : 1];
  auto request = [&] {
    if constexpr (XB > 0) {
#pragma unroll
      for (int b = 0; b < XB; ++b) request_x(min(k0 + b, a.DB - 1), raw[b]);
    }
  };
  if (a.E <= 128 && a.k <= 16)
    choose_all<Row, 16, 8>(a, ids, wts, flag, first, request);
  else if (a.E <= 256 && a.k <= 32)
    choose_all<Row, 32, 8>(a, ids, wts, flag, first, request);
  else
    choose_all<Row, 64, 16>(a, ids, wts, flag, first, request);
  lds_barrier();

  // Each wave makes the list: they write the same words, and need not wait again.
  int active = 0;
  for (int base = 0; base < a.E; base += 64) {
    const int e = base + lane;
    const int on = e < a.E ? flag[e] : 0;
    int sum;
    const int at = active + wave_prefix(on, &sum);
    if (on) {
      place[e] = at;
      list[at] = e;
    }
    active += sum;
  }
  wave_lds_sync();
  for (int i = lane; i < n; i += 64) {
    const int t = i / a.k;
    slots[place[ids[i]] * kTokens + t] = (uint8_t)(i - t * a.k);
  }
  wave_lds_sync();
  if (first) {
    for (int i = tid; i < fp8_tiles(a.dim); i += 64 * kWaves) a.count[i] = 0;
    if (tid == 0) a.head[0] = active;
    for (int i = tid; i < active; i += 64 * kWaves) a.head[1 + i] = list[i];
    for (int i = tid; i < active * (kTokens / 4); i += 64 * kWaves)
      a.head[1 + a.max_active + i] = lds[l.slots + i];
  }

  u32x4 xr[XB > 0 ? XB : 1][4][P];
  if constexpr (XB > 0) {
#pragma unroll
    for (int b = 0; b < XB; ++b) take_x(min(k0 + b, a.DB - 1), raw[b], xr[b]);
  }

  const int items = a.HB * 8 / kTiles;  // an expert's
  // One barrier an item: the sums of alternate items have LDS of their own, and half
  // of the waves finish an item while all go on to the next.
  int turn = 0;
  for (int item = blockIdx.x; item < active * items; item += gridDim.x, turn ^= 1) {
    const int at = item / items, nt0 = (item - at * items) * kTiles, nt = nt0 + sub;
    const int e = uniform_i32(list[at]);
    // a strip of 128 columns; a block past the wave's own is behind its end, and zeros
    const int64_t strip = ((int64_t)e * a.HB + nt / 8) * a.DB * (8 * kFp8Tile);
    const uint32_t in = (nt % 8) * kFp8Tile, end = (uint32_t)k1 * (8 * kFp8Tile);
    const rsrc_t gate_w = buffer(a.gate + strip, end), up_w = buffer(a.up + strip, end);
    const int64_t sc = ((int64_t)e * a.HB + nt / 8) * a.DB;
    f32x4 gs = {0.f, 0.f, 0.f, 0.f}, us = gs;
    auto add = [&](int kb, const Fp8Frag& gf, const Fp8Frag& uf, const u32x4 (&xf)[4][P]) {
      const f32x4 gp = block_sum<P>(gf, xf), up = block_sum<P>(uf, xf);
      const float sg = a.gate_s[sc + kb], su = a.up_s[sc + kb];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        gs[i] = fmaf(gp[i], sg, gs[i]);
        us[i] = fmaf(up[i], su, us[i]);
      }
    };
    if constexpr (XB > 0) {
      Fp8Frag gf[XB], uf[XB];
#pragma unroll
      for (int b = 0; b < XB; ++b) {
        gf[b] = load_tile(gate_w, lane, in + (k0 + b) * (8 * kFp8Tile));
        uf[b] = load_tile(up_w, lane, in + (k0 + b) * (8 * kFp8Tile));
      }
#pragma unroll
      for (int b = 0; b < XB; ++b) add(min(k0 + b, a.DB - 1), gf[b], uf[b], xr[b]);
    } else {
      for (int kb = k0; kb < k1; ++kb) {
        const Fp8Frag gf = load_tile(gate_w, lane, in + kb * (8 * kFp8Tile));
        const Fp8Frag uf = load_tile(up_w, lane, in + kb * (8 * kFp8Tile));
        u32x4 xf[4][P];
        request_x(kb, raw[0]);
        take_x(kb, raw[0], xf);
        add(kb, gf, uf, xf);
      }
    }
    float* p = part + turn * (kWaves * 2 * 256);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[(wave * 2 + 0) * 256 + i * 64 + lane] = gs[i];
      p[(wave * 2 + 1) * 256 + i * 64 + lane] = us[i];
    }
    __syncthreads();
    if ((wave >= kWaves / 2) == (turn == 1)) {
      const int id = tid & 255, t = id >> 4, c = id & 15;  // token and row of the tile
      const int src = (c & 3) * 64 + (c >> 2) * 16 + t;
      const int j = slots[at * kTokens + t];
      const int slot = t * a.k + j;
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int w = n * SHARE; w < (n + 1) * SHARE; ++w) {
          gate += p[(w * 2 + 0) * 256 + src];
          up += p[(w * 2 + 1) * 256 + src];
        }
        if (j != kNone)
          a.act[(int64_t)slot * (a.HB * 128) + fp8_column(nt0 + n, c >> 2) + (c & 3)] =
              silu(gate) * up * wts[slot];
      }
    }
  }
}

// Every wave of the call's `splits` workgroups a pair of tiles takes the blocks (e, b)
// with (e HB + b) mod (8 splits) of its number, 64 experts of the list at a time. A pair,
// so that a block of the activated rows, which is read from the caches and cut into its
// three operands by every wave that needs it, serves two tiles of weights: with one the
// layer took 86 us instead of 73 (sixteen tokens; fp32 rows of eight 66, 59). Rows of two
// bf16 parts, 18 bits, took 79 with one.
//
// The workgroup that finishes a tile's last split adds their sums up, in their order:
// splits write their sums past the caches, count themselves with an atomic, and only
// the last one goes on (nothing waits).
//
// What orders the sums before the count is the machine's rule, not the language's. On
// gfx950 an access of agent scope (sc1) goes past the XCD's L2 to where all eight meet: a
// store is acknowledged from there, and s_waitcnt vmcnt(0) waits for the acknowledgement,
// so the count is raised after the sums have arrived; the last split's loads are of agent
// scope too, and issued after the count's value came back. Agent fences would say this in
// the language, but they write back and discard the whole L2 of the XCD: tens of us.
template <typename Row>
__global__ void __launch_bounds__(64 * kWaves) layer_down_kernel(LayerArgs a, int splits) {
  extern __shared__ int head[];
  __shared__ f32x4 part[kWaves][2][64];
  const int lane = threadIdx.x & 63, wave = uniform_i32(threadIdx.x >> 6);
  const int pair = blockIdx.x / splits, split = blockIdx.x - pair * splits;
  const int t = lane & 15, g = lane >> 4;
  const int me = split * kWaves + wave, all = splits * kWaves;
  // the list and the slots, from kernel one
  const int words = 1 + a.max_active + a.max_active * (kTokens / 4);
  for (int i = threadIdx.x; i < words; i += 64 * kWaves) head[i] = a.head[i];
  __syncthreads();
  const int active = head[0];
  const int* list = head + 1;
  const uint8_t* slots = reinterpret_cast<const uint8_t*>(head + 1 + a.max_active);

  // A block's operands, requested while the block before is multiplied: without
  // branches, so that waiting for the one does not wait for the other. What is not
  // there (no block, a token that did not choose the expert) lies behind its buffer's
  // end and arrives as zeros.
  struct Unit {
    Fp8Frag w[2];
    u32x4 x[4][2];  // 8 fp32 values of each step
    float scale;
    bool on, live;
  };
  const rsrc_t act = buffer(a.act, a.act_bytes);
  const uint32_t row_bytes = (uint32_t)a.HB * 512;
  int base = 0, mine = 0, first = 0, at = 0, e = 0, b = a.HB;
  uint64_t hits = 0;
  bool more = active > 0;
  auto look = [&] {  // the wave's experts among the 64 from base on
    mine = base + lane < active ? list[base + lane] : 0;
    first = (int)(((uint32_t)(me - mine * a.HB) + (uint32_t)all * (uint32_t)a.HB * kMaxExperts) %
                  (uint32_t)all);
    hits = __ballot(base + lane < active && first < a.HB);
  };
  auto next = [&] {  // the wave's next block, or more = false
    b += all;
    while (b >= a.HB) {
      if (!hits) {
        base += 64;
        if (base >= active) {
          more = false;
          return;
        }
        look();
        continue;
      }
      const int l = __builtin_ctzll(hits);
      hits &= hits - 1;
      at = base + l;
      e = __builtin_amdgcn_readlane(mine, l);
      b = __builtin_amdgcn_readlane(first, l);
    }
  };
  auto request = [&](Unit& u) {
    if (more) next();
    u.live = more;
    const int64_t strip = (int64_t)e * a.DB + pair / 4;
    const rsrc_t w = buffer(a.down + strip * a.HB * (8 * kFp8Tile), more ? a.HB * (8 * kFp8Tile) : 0);
    const int in_strip = more ? b : 0;
#pragma unroll
    for (int n = 0; n < 2; ++n)
      u.w[n] = load_tile(w, lane, (in_strip * 8 + pair % 4 * 2 + n) * kFp8Tile);
    u.scale = a.down_s[strip * a.HB + in_strip];
    const int j = slots[at * kTokens + t];
    u.on = j != kNone;
    const uint32_t x = u.on && more ? (uint32_t)(t * a.k + j) * row_bytes + g * 128 : 0xffff0000u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        u.x[i][h] = buffer_load16(act, x, in_strip * 512 + i * 32 + h * 16);
  };
  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  auto add = [&](const Unit& u) {
    u32x4 x[4][3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
      F32Row::widen16(u.x[i][0], v);
      F32Row::widen16(u.x[i][1], v + 4);
      split8<3>(v, x[i]);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const f32x4 s = block_sum<3>(u.w[n], x);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = u.on ? fmaf(s[i], u.scale, acc[n][i]) : acc[n][i];
    }
  };
  if (more) look();
  Unit u0, u1;
  request(u0);
  while (u0.live) {
    request(u1);
    add(u0);
    if (!u1.live) break;
    request(u0);
    add(u1);
  }
#pragma unroll
  for (int n = 0; n < 2; ++n) part[wave][n][lane] = acc[n];
  __syncthreads();
  if (wave > 1) return;
  // waves 0 and 1 finish a tile each
  const int nt = 2 * pair + wave;
  f32x4 sum = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += part[w][wave][lane];
  if (splits > 1) {
    float* sums = a.sums + (int64_t)nt * splits * 256;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __hip_atomic_store(&sums[split * 256 + i * 64 + lane], sum[i], __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_AGENT);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt 0: the sums are where every XCD sees them
    int done = 0;
    if (lane == 0)
      done = __hip_atomic_fetch_add(&a.count[nt], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (uniform_i32(done) != splits - 1) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    sum = f32x4{0.f, 0.f, 0.f, 0.f};
    constexpr int kTogether = 4;  // splits whose sums are on their way together
    for (int s0 = 0; s0 < splits; s0 += kTogether) {
      f32x4 v[kTogether];
#pragma unroll
      for (int j = 0; j < kTogether; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[j][i] = __hip_atomic_load(&sums[min(s0 + j, splits - 1) * 256 + i * 64 + lane],
                                      __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int j = 0; j < kTogether; ++j)
        if (s0 + j < splits) sum += v[j];
    }
  }
  if (t >= a.T) return;
  const int n = fp8_column(nt, g);
  typename Row::elem* p = static_cast<typename Row::elem*>(a.out) + (int64_t)t * a.out_ld + n;
  typedef typename Row::elem elem;
  if (n + 4 <= a.dim) {
    if constexpr (sizeof(elem) == 2) {
      *reinterpret_cast<u32x2_any*>(p) = u32x2{pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
    } else {
      *reinterpret_cast<u32x4_any*>(p) = __builtin_bit_cast(u32x4, sum);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (n + i < a.dim) p[i] = Row::narrow(sum[i]);
  }
}

// Splits of the down product's blocks, so that there is a workgroup a CU, as long as
// each of their waves has a block. 64 pairs of tiles in 2, 4, 8 splits, the layer, us: two
// tokens 28.2, 25.6, 28.5; sixteen 92, 74, 78; 224 pairs (dim 7168) in 1, 2, 4: 98, 101,
// 109. Narrow rows have few pairs (154 columns: 8 splits 30, 32 24.8).
int splits_of(int64_t T, int64_t E, int64_t k, int64_t dim, int64_t hidden) {
  const int64_t pairs = fp8_tiles((int32_t)dim) / 2;
  const int64_t blocks = std::min(E, T * k) * ((hidden + 127) / 128);
  int s = 1;
  while (s < 32 && pairs * s < 256 && blocks >= 2 * s * kWaves) s *= 2;
  return s;
}

struct LayerSpace {
  int64_t count, sums, act, total;  // bytes
};
LayerSpace space_of(int64_t T, int64_t E, int64_t k, int64_t dim, int64_t hidden) {
  const int64_t active = std::min(E, T * k), width = (hidden + 127) / 128 * 128;
  const int64_t tiles = fp8_tiles((int32_t)dim);
  auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
  LayerSpace s{};
  s.count = up((1 + active + active * (kTokens / 4)) * 4);
  s.sums = s.count + up(tiles * 4);
  s.act = s.sums + tiles * splits_of(T, E, k, dim, hidden) * 1024;
  s.total = s.act + T * k * width * 4;
  return s;
}

int32_t check_layer(const char* who, int64_t n_tokens, int32_t n_experts, int32_t top_k,
                    int32_t dim, int32_t hidden) {
  if (n_tokens < 0 || n_tokens > kTokens)
    return fail(MLORA_ERR_INVALID, "%s: n_tokens=%lld outside [0, %d]", who, (long long)n_tokens,
                kTokens);
  if (n_experts < 1 || n_experts > kMaxExperts)
    return fail(MLORA_ERR_INVALID, "%s: n_experts=%d outside [1, %d]", who, n_experts, kMaxExperts);
  if (top_k < 1 || top_k > n_experts || top_k > kMaxTopK)
    return fail(MLORA_ERR_INVALID, "%s: top_k=%d outside [1, min(n_experts=%d, %d)]", who, top_k,
                n_experts, kMaxTopK);
  if (dim < 1 || dim > kFp8MaxDim || hidden < 1 || hidden > kFp8MaxDim)
    return fail(MLORA_ERR_INVALID, "%s: dim=%d, hidden=%d outside [1, %d]", who, dim, hidden,
                kFp8MaxDim);
  // the activated rows are read with 32-bit offsets
  if (n_tokens * top_k * 4 * (((int64_t)hidden + 127) / 128 * 128) >= 0xff000000ll)
    return fail(MLORA_ERR_INVALID, "%s: hidden=%d is too wide for %lld rows", who, hidden,
                (long long)(n_tokens * top_k));
  return MLORA_OK;
}

template <typename Row, int XB, int SHARE>
void launch_gate_up_as(const LayerArgs& a, hipStream_t s) {
  const Lds l = lds_of(a.T * a.k, a.E, a.max_active);
  const int64_t items = (int64_t)a.max_active * a.HB * SHARE;
  // As many workgroups as are there at once: two a CU (a SIMD holds four of their waves'
  // registers), one where a wave keeps more than 48 registers of x, with which it holds two
  // or three. More would choose the experts again. Sixteen tokens, 256, 512, 768, 1024: the layer 85, 82, 93, 95 us; one fp32 token
  // of 1834 -> 1010, 256 and 512: 25, 30.
  constexpr int kXRegs = XB * (sizeof(typename Row::elem) == 2 ? 16 : 48);
  hipLaunchKernelGGL((layer_gate_up_kernel<Row, XB, SHARE>),
                     dim3((unsigned)std::min<int64_t>(items, kXRegs > 48 ? 256 : 512)),
                     dim3(64 * kWaves), l.total * 4, s, a);
}

template <typename Row>
void launch_gate_up(const LayerArgs& a, hipStream_t s) {
  const int blocks = (a.DB + kWaves - 1) / kWaves;  // a wave's
  constexpr bool kBf16 = sizeof(typename Row::elem) == 2;
  if (a.DB == 1) return launch_gate_up_as<Row, 1, 1>(a, s);
  if (a.DB == 2) return launch_gate_up_as<Row, 1, 2>(a, s);
  if (a.DB <= 4) return launch_gate_up_as<Row, 1, 4>(a, s);
  if (blocks <= 1) return launch_gate_up_as<Row, 1, 8>(a, s);
  if (blocks <= 2) return launch_gate_up_as<Row, 2, 8>(a, s);
  if (kBf16 && blocks <= 4) return launch_gate_up_as<Row, kBf16 ? 4 : 0, 8>(a, s);
  launch_gate_up_as<Row, 0, 8>(a, s);
}

template <typename Row>
int32_t launch_layer(const char* who, const LayerArgs& a, hipStream_t s) {
  launch_gate_up<Row>(a, s);
  if (int32_t rc = launch_status(who)) return rc;
  const int splits = splits_of(a.T, a.E, a.k, a.dim, a.hidden);
  hipLaunchKernelGGL((layer_down_kernel<Row>), dim3(fp8_tiles(a.dim) / 2 * splits), dim3(64 * kWaves),
                     (1 + a.max_active + a.max_active * (kTokens / 4)) * 4, s, a, splits);
  return launch_status(who);
}

}  // namespace
}  // namespace mlora

using namespace mlora;

extern "C" uint64_t mlora_moe_layer_workspace_bytes(int64_t n_tokens, int32_t n_experts,
                                                    int32_t top_k, int32_t dim, int32_t hidden) {
  if (check_layer("mlora_moe_layer_workspace_bytes", n_tokens, n_experts, top_k, dim, hidden))
    return 0;
  return n_tokens == 0 ? 0 : (uint64_t)space_of(n_tokens, n_experts, top_k, dim, hidden).total;
}

extern "C" int32_t mlora_moe_layer(const mlora_fp8_route* gate, const mlora_fp8_route* up,
                                   const mlora_fp8_route* down, const void* x, int64_t x_ld,
                                   int32_t dtype, int64_t n_tokens, const void* logits,
                                   int64_t logits_ld, int32_t top_k, int32_t renormalize,
                                   void* out, int64_t out_ld, int32_t* indices, float* weights,
                                   void* workspace, uint64_t workspace_bytes, void* stream) {
  const char* who = "mlora_moe_layer";
  if (int32_t rc = check_fp8_route(who, "gate", gate)) return rc;
  if (int32_t rc = check_fp8_route(who, "up", up)) return rc;
  if (int32_t rc = check_fp8_route(who, "down", down)) return rc;
  if (gate->n_experts != up->n_experts || gate->n_experts != down->n_experts ||
      gate->k_in != up->k_in || gate->n_out != up->n_out || down->k_in != gate->n_out ||
      down->n_out != gate->k_in)
    return fail(MLORA_ERR_INVALID, "%s: the routes' sizes do not fit each other", who);
  if (dtype != MLORA_BF16 && dtype != MLORA_F32)
    return fail(MLORA_ERR_INVALID, "%s: dtype %d is neither bf16 nor f32", who, dtype);
  const int32_t E = gate->n_experts, dim = gate->k_in, hidden = gate->n_out;
  if (int32_t rc = check_layer(who, n_tokens, E, top_k, dim, hidden)) return rc;
  if (x_ld < dim || out_ld < dim || logits_ld < E)
    return fail(MLORA_ERR_INVALID, "%s: row stride below the row's width", who);
  if (n_tokens == 0) {
    clear_error();
    return MLORA_OK;
  }
  if (!x || !logits || !out) return fail(MLORA_ERR_INVALID, "%s: NULL pointer", who);
  const LayerSpace sp = space_of(n_tokens, E, top_k, dim, hidden);
  if (!workspace || workspace_bytes < (uint64_t)sp.total)
    return fail(MLORA_ERR_CAPACITY, "%s: workspace of %llu bytes, %lld needed", who,
                (unsigned long long)(workspace ? workspace_bytes : 0), (long long)sp.total);
  if (!aligned(workspace, 256))
    return fail(MLORA_ERR_INVALID, "%s: workspace must be 256-byte aligned", who);
  LayerArgs a{};
  a.logits = logits;
  a.logits_ld = logits_ld;
  a.x = x;
  a.x_ld = x_ld;
  a.gate = static_cast<const uint8_t*>(gate->weights);
  a.up = static_cast<const uint8_t*>(up->weights);
  a.down = static_cast<const uint8_t*>(down->weights);
  a.gate_s = static_cast<const float*>(gate->scales);
  a.up_s = static_cast<const float*>(up->scales);
  a.down_s = static_cast<const float*>(down->scales);
  a.out = out;
  a.out_ld = out_ld;
  a.indices = indices;
  a.weights = weights;
  a.head = static_cast<int32_t*>(workspace);
  a.count = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + sp.count);
  a.sums = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sp.sums);
  a.act = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sp.act);
  a.act_bytes = (uint32_t)(sp.total - sp.act);
  a.T = (int32_t)n_tokens;
  a.E = E;
  a.k = top_k;
  a.renorm = renormalize;
  a.dim = dim;
  a.hidden = hidden;
  a.DB = (dim + 127) / 128;
  a.HB = (hidden + 127) / 128;
  a.max_active = std::min(E, a.T * top_k);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  return dtype == MLORA_BF16 ? launch_layer<Bf16Row>(who, a, s)
                             : launch_layer<F32Row>(who, a, s);
}
