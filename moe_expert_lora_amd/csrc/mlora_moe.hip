// The MoE layer's row work around the fold, for gfx950 (MI355X): the router's
// top-k choice and its gradient, the stable sort of the routed (token, slot)
// rows by expert, the dispatch of token rows to sorted rows, and the weighted
// combine of expert rows with its gradient.
#include "mlora_router.h"

namespace mlora {
namespace {

// ---------------------------------------------------------------------------
// router
// ---------------------------------------------------------------------------
//
// The choice itself is in mlora_router.h; lanes 0 .. k - 1 of a token write the
// results.

struct RouterArgs {
  const void* logits;
  int64_t ld;
  int32_t* indices;
  float* weights;
  const float* d_weights;  // backward
  void* d_logits;
  int64_t d_ld;
  int32_t n_tokens;
  int32_t E;
  int32_t k;
  int32_t renorm;
};

// A kernel's leading plain arguments arrive in registers at its start; what is
// needed for the first loads is passed there, and the struct, which is read
// from memory, for the rest.
__device__ __forceinline__ void set_lead(RouterArgs& a, const void* logits, int64_t ld,
                                         int32_t n_tokens, int32_t E, int32_t k, int32_t renorm) {
  a.logits = logits;
  a.ld = ld;
  a.n_tokens = n_tokens;
  a.E = E;
  a.k = k;
  a.renorm = renorm;
}

template <typename Row, int LPT, int VPL, int VEC, bool WIDE>
__global__ void __launch_bounds__(256) router_topk_kernel(const void* logits, int64_t ld, int32_t n_tokens, int32_t E,
                                                          int32_t k, int32_t renorm, RouterArgs a) {
  set_lead(a, logits, ld, n_tokens, E, k, renorm);
  const int gl = threadIdx.x & (LPT - 1);
  const int token = flat_group() * (int)(blockDim.x / LPT) + (int)(threadIdx.x / LPT);
  const bool on = token < a.n_tokens;  // lanes past the end stay for the reductions
  float v[VPL];
  load_row<Row, LPT, VPL, VEC, WIDE>(a.logits, (int64_t)(on ? token : 0) * a.ld, a.E, gl, v);
  int mine_e;
  const float w = choose_experts<Row, LPT, VPL, VEC>(v, a.E, a.k, a.renorm, gl, &mine_e);
  if (on && gl < a.k) {
    a.indices[(int64_t)token * a.k + gl] = mine_e;
    a.weights[(int64_t)token * a.k + gl] = w;
  }
}

// Gradient of the weights with respect to the logits, p recomputed:
//   dl_e = p_e (dw_e - dot), dot = sum_sel dw p            (softmax over all)
//   dl_e = w_e (dw_e - dot) on the chosen experts, else 0  (renormalised: the
//          weights are a softmax over the chosen logits alone)
// dw_e reaches expert e's lane through a row of LDS; a word no dw has marks
// the experts that were not chosen.
template <typename Row, int LPT, int VPL, int VEC, bool WIDE>
__global__ void __launch_bounds__(256) router_backward_kernel(const void* logits, int64_t ld, int32_t n_tokens,
                                                              int32_t E, int32_t k, int32_t renorm,
                                                              RouterArgs a) {
  set_lead(a, logits, ld, n_tokens, E, k, renorm);
  constexpr uint32_t kUnset = 0xffffffffu;
  __shared__ uint32_t lds[256 / LPT][LPT * VPL];
  const int gl = threadIdx.x & (LPT - 1);
  const int token = flat_group() * (int)(blockDim.x / LPT) + (int)(threadIdx.x / LPT);
  const bool on = token < a.n_tokens;
  const int64_t t = on ? token : 0;
  uint32_t* s = lds[threadIdx.x / LPT];
  float v[VPL];
  load_row<Row, LPT, VPL, VEC, WIDE>(a.logits, t * a.ld, a.E, gl, v);
  int e_dw = -1;
  uint32_t dw_bits = 0;
  if (gl < a.k) {
    e_dw = a.indices[t * a.k + gl];
    dw_bits = __float_as_uint(a.d_weights[t * a.k + gl]);
    if ((dw_bits & 0x7fffffffu) > 0x7f800000u) dw_bits = 0x7fc00000u;
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) s[expert_of<LPT, VEC>(j, gl)] = kUnset;
  wave_lds_sync();
  if (e_dw >= 0 && e_dw < a.E) s[e_dw] = dw_bits;
  wave_lds_sync();
  uint32_t d[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) d[j] = s[expert_of<LPT, VEC>(j, gl)];

  // the maximum and the sum of the softmax, over all or over the chosen
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const bool in = expert_of<LPT, VEC>(j, gl) < a.E && (!a.renorm || d[j] != kUnset);
    m = max(m, in ? order_key(__float_as_uint(v[j])) : 0u);
  }
  m = group_max<LPT>(m);
  const float top = m == 0 ? kNegInf : key_value(m);
  float sum = 0.f, dot = 0.f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const bool in = expert_of<LPT, VEC>(j, gl) < a.E && (!a.renorm || d[j] != kUnset);
    v[j] = in ? expf(v[j] - top) : 0.f;
    sum += v[j];
    if (d[j] != kUnset) dot += __uint_as_float(d[j]) * v[j];
  }
  sum = group_sum<LPT>(sum);
  dot = group_sum<LPT>(dot) / sum;
  if (!on) return;
  typename Row::elem* out = static_cast<typename Row::elem*>(a.d_logits) + t * a.d_ld;
#pragma unroll
  for (int j = 0; j < VPL; j += VEC) {
    const int e = expert_of<LPT, VEC>(j, gl);
    float g[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float dw = d[j + i] != kUnset ? __uint_as_float(d[j + i]) : 0.f;
      const bool zero = top == kNegInf || (a.renorm && d[j + i] == kUnset);
      g[i] = zero ? 0.f : v[j + i] / sum * (dw - dot);
    }
    if constexpr (!WIDE) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (e + i < a.E) out[e + i] = Row::narrow(g[i]);
    } else {
      if (e < a.E) {
        typedef typename Row::elem vec __attribute__((ext_vector_type(VEC)));
        vec w;
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = Row::narrow(g[i]);
        *reinterpret_cast<vec*>(out + e) = w;
      }
    }
  }
}

template <typename Row, int LPT, int VPL, int VEC, bool WIDE>
void launch_router(const RouterArgs& a, bool backward, hipStream_t s) {
  // Small batches get workgroups of one wave, so that their few tokens spread
  // over the CUs; large ones four waves.
  const int64_t lanes = (int64_t)a.n_tokens * LPT;
  const int threads = lanes < 64 * 1024 ? 64 : 256;
  const dim3 grid = flat_grid((lanes + threads - 1) / threads);
  if (backward)
    hipLaunchKernelGGL((router_backward_kernel<Row, LPT, VPL, VEC, WIDE>), grid, dim3(threads), 0, s,
                       a.logits, a.ld, a.n_tokens, a.E, a.k, a.renorm, a);
  else
    hipLaunchKernelGGL((router_topk_kernel<Row, LPT, VPL, VEC, WIDE>), grid, dim3(threads), 0, s,
                       a.logits, a.ld, a.n_tokens, a.E, a.k, a.renorm, a);
}

// Lanes per token and values per lane: 16 lanes hold up to 128 experts (four
// tokens a wave; the reductions stay in rows of 16), 32 up to 256, a wave up to
// 1024; top_k winners need as many lanes. Fewer lanes with more values save
// instructions where tokens fill the chip and cost latency where they do not.
// 256 experts, top 8, choice and gradient together, us: 8192 tokens of fp32 in
// 16, 32, 64 lanes 12.6, 12.1, 13.7; 80 tokens 9.1, 7.2, 7.2. 512 experts in 32
// lanes 19.6 and 9.6, in 64 20.0 and 7.3.
template <typename Row, bool WIDE>
void dispatch_router(const RouterArgs& a, bool backward, hipStream_t s) {
  constexpr int V = Row::kPer16;
  if (a.E <= 128 && a.k <= 16) return launch_router<Row, 16, 8, V, WIDE>(a, backward, s);
  if (a.E <= 256 && a.k <= 32) return launch_router<Row, 32, 8, V, WIDE>(a, backward, s);
  if (a.E <= 512) return launch_router<Row, 64, 8, V, WIDE>(a, backward, s);
  launch_router<Row, 64, 16, V, WIDE>(a, backward, s);
}

int32_t run_router(const RouterArgs& a, int32_t dtype, bool backward, const char* who,
                   hipStream_t s) {
  const int es = dtype == MLORA_BF16 ? 2 : 4;
  const int v = 16 / es;
  const bool vec = a.E % v == 0 && a.ld % v == 0 && aligned(a.logits, 16) &&
                   (!backward || (a.d_ld % v == 0 && aligned(a.d_logits, 16)));
  (void)hipGetLastError();
  if (dtype == MLORA_BF16) {
    if (vec)
      dispatch_router<Bf16Row, true>(a, backward, s);
    else
      dispatch_router<Bf16Row, false>(a, backward, s);
  } else {
    if (vec)
      dispatch_router<F32Row, true>(a, backward, s);
    else
      dispatch_router<F32Row, false>(a, backward, s);
  }
  return launch_status(who);
}

int32_t check_router(const char* who, int32_t dtype, int64_t n_tokens, int32_t n_experts,
                     int32_t top_k, int64_t ld) {
  if (dtype != MLORA_BF16 && dtype != MLORA_F32)
    return fail(MLORA_ERR_INVALID, "%s: dtype %d is neither bf16 nor f32", who, dtype);
  if (n_tokens < 0 || n_tokens > kMaxRows)
    return fail(MLORA_ERR_INVALID, "%s: n_tokens=%lld out of range", who, (long long)n_tokens);
  if (n_experts < 1 || n_experts > kMaxExperts)
    return fail(MLORA_ERR_INVALID, "%s: n_experts=%d outside [1, %d]", who, n_experts,
                kMaxExperts);
  if (top_k < 1 || top_k > n_experts || top_k > kMaxTopK)
    return fail(MLORA_ERR_INVALID, "%s: top_k=%d outside [1, min(n_experts=%d, %d)]", who, top_k,
                n_experts, kMaxTopK);
  if (ld < n_experts)
    return fail(MLORA_ERR_INVALID, "%s: row stride %lld below n_experts=%d", who, (long long)ld,
                n_experts);
  return MLORA_OK;
}

// ---------------------------------------------------------------------------
// sort by expert
// ---------------------------------------------------------------------------
//
// A stable counting sort of the flat (token, slot) ids by expert; ids outside
// [0, E) go into a last bucket E, whose sorted places are written as -1. A
// tile of 1024 R ids is split over 16 waves in runs of 64 R. A wave goes
// through its run 64 ids at a time: lanes with the same key find each other
// by one ballot per key bit, their rank is the number of such lanes before
// them plus the wave's count of the key so far (LDS). A prefix over the waves
// and over the keys then turns ranks into places. All sums are integers, so
// the result does not depend on any order.
//
// Up to 1024 ids run as one workgroup. Up to kSortOne, each workgroup places
// 1024 ids and counts every id itself for the places before its own. More take
// two kernels: counts per block into the workspace, then each block sums the
// counts before it (and all of them) itself and places its ids.
//
// Measured (128 experts, skewed, us a call; a launch alone is 2.3 to 3): 4096
// ids recounted 4.6, in two kernels 9.0; 32768: 7.9 and 10.1; 49152: 9.7 and
// 10.2; 65536: 11.6 and 10.5. What bounds the recount is LDS atomics, one per
// id and workgroup; the two kernels, their two starts.

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortR = 4;                       // ids per thread of a tile
constexpr int kSortTile = kSortThreads * kSortR;
constexpr int64_t kSortOne = 40960;             // ids of the one-kernel form
constexpr int kSortBlocks = 256;                // most blocks of the two-kernel form

struct SortArgs {
  const int32_t* ids;
  int32_t* offsets;
  int32_t* sorted_ids;
  int32_t* slot_rows;
  int32_t* counts;  // workspace [blocks][E + 1]
  int32_t n;
  int32_t E;
  int32_t key_bits;
  int32_t blocks;
  int32_t tiles_per_block;
};

__device__ __forceinline__ int sort_key(int id, int E) {
  return (uint32_t)id < (uint32_t)E ? id : E;
}

// Lanes of the wave with this lane's key (every lane active).
__device__ __forceinline__ uint64_t match_key(int key, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    m &= ((key >> b) & 1) ? set : ~set;
  }
  return m;
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
  extern __shared__ int cnt[];
  const int nk = a.E + 1;
  for (int e = threadIdx.x; e < nk; e += kSortThreads) cnt[e] = 0;
  __syncthreads();
  const int64_t per = (int64_t)a.tiles_per_block * kSortTile;
  const int64_t lo = blockIdx.x * per;
  const int64_t hi = lo + per < a.n ? lo + per : a.n;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads)
    atomicAdd(&cnt[sort_key(a.ids[i], a.E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < nk; e += kSortThreads)
    a.counts[(int64_t)blockIdx.x * nk + e] = cnt[e];
}

// LDS: base[nk] (where the block's next id of a key goes), total[nk] (the
// call's counts), tile_cnt[nk], then 16-bit counts [kSortWaves][nk] (a tile
// has 64 R ids a wave and 1024 R in all).
size_t sort_lds_bytes(int E) { return (size_t)(E + 1) * (3 * 4 + kSortWaves * 2); }

__global__ void __launch_bounds__(256) sort_empty_kernel(SortArgs a) {
  for (int e = threadIdx.x; e <= a.E; e += 256) a.offsets[e] = 0;
}

// How a block learns the counts of the ids before its own, and of all.
enum SortMode {
  kSortAlone,    // one block: its tile's counts
  kSortRecount,  // it counts every id itself (a tile per block)
  kSortCounted   // sort_count_kernel's counts
};
constexpr int kSortCopies = 4;  // of each counter in kSortRecount: fewer lanes on one address

template <int R, SortMode MODE>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const int32_t* ids, int32_t n, int32_t E,
                                                              int32_t key_bits, SortArgs a) {
  a.ids = ids;
  a.n = n;
  a.E = E;
  a.key_bits = key_bits;
  extern __shared__ int lds[];
  __shared__ int wave_sum[kSortWaves];
  const int nk = a.E + 1, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int* base = lds;
  int* total = lds + nk;
  int* tile_cnt = lds + 2 * nk;
  uint16_t* waves = reinterpret_cast<uint16_t*>(lds + 3 * nk);
  uint16_t* mine = waves + wave * nk;
  constexpr int kTile = kSortThreads * R;
  if constexpr (MODE == kSortRecount) {
    // counters [before this tile, not before][copy][key], over the whole LDS
    // of the later steps
    for (int i = tid; i < 2 * kSortCopies * nk; i += kSortThreads) lds[i] = 0;
    __syncthreads();
    const int t0 = (int)blockIdx.x * kTile, whole = a.n & ~3;
    int* mycopy = lds + (lane & (kSortCopies - 1)) * nk;
    for (int i = tid * 4; i < whole; i += kSortThreads * 4) {
      const int4 id = *reinterpret_cast<const int4*>(a.ids + i);
      int* c = mycopy + (i < t0 ? 0 : kSortCopies * nk);  // t0 is a multiple of 4
      atomicAdd(&c[sort_key(id.x, a.E)], 1);
      atomicAdd(&c[sort_key(id.y, a.E)], 1);
      atomicAdd(&c[sort_key(id.z, a.E)], 1);
      atomicAdd(&c[sort_key(id.w, a.E)], 1);
    }
    if (tid < a.n - whole) {
      const int i = whole + tid;
      atomicAdd(&mycopy[(i < t0 ? 0 : kSortCopies * nk) + sort_key(a.ids[i], a.E)], 1);
    }
    __syncthreads();
    int before[2], all[2];  // of keys tid and tid + 1024
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = tid + h * kSortThreads;
      before[h] = all[h] = 0;
      if (e < nk) {
#pragma unroll
        for (int c = 0; c < kSortCopies; ++c) {
          before[h] += lds[c * nk + e];
          all[h] += lds[(kSortCopies + c) * nk + e];
        }
        all[h] += before[h];
      }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = tid + h * kSortThreads;
      if (e < nk) {
        base[e] = before[h];
        total[e] = all[h];
      }
    }
  } else {
    for (int e = tid; e < 2 * nk; e += kSortThreads) lds[e] = 0;
  }
  if constexpr (MODE == kSortCounted) {
    __syncthreads();
    const int parts = kSortThreads > nk ? kSortThreads / nk : 1;
    for (int i = tid; i < parts * nk; i += kSortThreads) {
      const int part = i / nk, e = i - part * nk;
      int before = 0, all = 0;
      for (int b = part; b < a.blocks; b += parts) {
        const int c = a.counts[(int64_t)b * nk + e];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
      atomicAdd(&base[e], before);
      atomicAdd(&total[e], all);
    }
  }
  for (int tile = 0; tile < a.tiles_per_block; ++tile) {
    const int64_t t0 = ((int64_t)blockIdx.x * a.tiles_per_block + tile) * kTile;
    if (t0 >= a.n) break;
    int id[R], key[R], rank[R];
    const int64_t first = t0 + (int64_t)wave * 64 * R + lane;
#pragma unroll
    for (int r = 0; r < R; ++r) id[r] = first + r * 64 < a.n ? a.ids[first + r * 64] : -1;
    for (int e = lane; e < nk; e += 64) mine[e] = 0;
    wave_lds_sync();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool in = first + r * 64 < a.n;
      key[r] = in ? sort_key(id[r], a.E) : nk;  // nk: past the end, no bucket
      const uint64_t same = match_key(key[r], a.key_bits);
      const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32),
                                                   __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0u));
      const int old = in ? mine[key[r]] : 0;
      rank[r] = old + before;
      wave_lds_sync();
      if (in && before == 0) mine[key[r]] = (uint16_t)(old + __popcll(same));
      wave_lds_sync();
    }
    __syncthreads();
    for (int e = tid; e < nk; e += kSortThreads) {
      int run = 0;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        const int c = waves[w * nk + e];
        waves[w * nk + e] = (uint16_t)run;
        run += c;
      }
      tile_cnt[e] = run;
      if (MODE == kSortAlone) total[e] = run;
    }
    __syncthreads();
    if (tile == 0) {
      // exclusive prefix of `total` over the experts, a thread each (E <= 1024);
      // the dropped ones' bucket E starts behind them all
      int sum;
      int at = wave_prefix(tid < a.E ? total[tid] : 0, &sum);
      if (lane == 0) wave_sum[wave] = sum;
      __syncthreads();
      int live = 0;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        at += w < wave ? wave_sum[w] : 0;
        live += wave_sum[w];
      }
      if (tid < a.E) {
        base[tid] += at;
        if (blockIdx.x == 0) a.offsets[tid] = at;
      }
      if (tid == 0) {
        base[a.E] += live;
        if (blockIdx.x == 0) a.offsets[a.E] = live;
      }
      __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t i = first + r * 64;
      if (i < a.n) {
        const int pos = base[key[r]] + mine[key[r]] + rank[r];
        const bool live = key[r] < a.E;
        a.sorted_ids[pos] = live ? (int)i : -1;
        a.slot_rows[i] = live ? pos : -1;
      }
    }
    if (tile + 1 < a.tiles_per_block) {
      __syncthreads();
      for (int e = tid; e < nk; e += kSortThreads) base[e] += tile_cnt[e];
      __syncthreads();
    }
  }
}

// Blocks that count ahead in the two-kernel form (0: one kernel).
int sort_blocks(int64_t n) {
  if (n <= kSortOne) return 0;
  const int64_t tiles = (n + kSortTile - 1) / kSortTile;
  const int64_t per = (tiles + kSortBlocks - 1) / kSortBlocks;
  return (int)((tiles + per - 1) / per);
}

// ---------------------------------------------------------------------------
// dispatch, combine and the combine's gradient
// ---------------------------------------------------------------------------
//
// G threads own one token and go through its columns 16 bytes (or one
// element, where a row's start or width does not allow 16) at a time. A
// token's top_k slots are taken kSlots at a time: their row numbers are read
// once, and the slots' loads are all in flight together. Dispatch reads each
// x row once and writes it to the token's sorted rows; combine sums its rows
// in slot order in fp32 and rounds once; the gradient keeps kSlots dot
// products per thread and adds them up over the G threads in a fixed order.
// Rows that no slot names (sorted_ids < 0: the places after the last live
// one) are written as zeros by the token whose flat ids t * k + j they have
// as row numbers, so every row is written exactly once.

constexpr int kSlots = 8;

struct RowsArgs {
  const void* src;        // dispatch: x; combine: rows; gradient: rows
  int64_t src_ld;
  const void* d_out;      // gradient
  int64_t d_out_ld;
  void* dst;              // dispatch: out rows; combine: out; gradient: d_rows
  int64_t dst_ld;
  const float* weights;   // [n_tokens * k] or null (1)
  const int32_t* slot_rows;
  const int32_t* sorted_ids;
  float* d_weights;
  int64_t n_rows;
  int32_t n_tokens;
  int32_t k;
  int32_t units;          // columns per row, in loads
};

// One load of a row: 16 bytes, or one element.
template <typename Row, bool WIDE>
struct Unit {
  static constexpr int kN = Row::kPer16;
  typedef u32x4 raw;
  static __device__ __forceinline__ raw zero() { return u32x4{0, 0, 0, 0}; }
  static __device__ __forceinline__ void widen(raw v, float* f) { Row::widen16(v, f); }
  static __device__ __forceinline__ raw narrow(const float* f) { return Row::narrow16(f); }
};
template <typename Row>
struct Unit<Row, false> {
  static constexpr int kN = 1;
  typedef typename Row::elem raw;
  static __device__ __forceinline__ raw zero() { return 0; }
  static __device__ __forceinline__ void widen(raw v, float* f) { f[0] = Row::widen(v); }
  static __device__ __forceinline__ raw narrow(const float* f) { return Row::narrow(f[0]); }
};

template <typename Row, typename U>
__device__ __forceinline__ U* row_at(const void* base, int64_t row, int64_t ld) {
  typedef typename Row::elem elem;
  return reinterpret_cast<U*>(const_cast<elem*>(static_cast<const elem*>(base)) + row * ld);
}

// Rows go past the caches' keep: each is read or written once, and k times as
// many of them move as of tokens' rows (32768 rows of 4 KB: dispatch 32.5 -> 27.4
// us, combine 31.4 -> 26.5, its gradient on 16384 rows of 8 KB 62.4 -> 55.3; no
// difference at 640 rows).
template <typename T>
__device__ __forceinline__ T load_once(const T* p) {
  return __builtin_nontemporal_load(p);
}
template <typename T>
__device__ __forceinline__ void store_once(T* p, T v) {
  __builtin_nontemporal_store(v, p);
}

// p's entries of slots j0 .. j0 + kSlots - 1 of token t, all requested together
// (places past the last slot read the last one).
__device__ __forceinline__ void slot_entries(const int32_t* p, const RowsArgs& a, int t, int j0,
                                             int (&v)[kSlots]) {
  p += (int64_t)t * a.k + j0;
  const int last = a.k - 1 - j0;
#pragma unroll
  for (int j = 0; j < kSlots; ++j) v[j] = p[min(j, last)];
}

// Row numbers of slots j0 .. j0 + kSlots - 1 of token t; -1 where there is none.
__device__ __forceinline__ void slot_numbers(const RowsArgs& a, int t, int j0,
                                             int (&row)[kSlots]) {
  if (a.slot_rows) {
    slot_entries(a.slot_rows, a, t, j0, row);
  } else {
#pragma unroll
    for (int j = 0; j < kSlots; ++j) row[j] = t * a.k + j0 + j;
  }
#pragma unroll
  for (int j = 0; j < kSlots; ++j)
    if (j0 + j >= a.k || (uint32_t)row[j] >= (uint64_t)a.n_rows) row[j] = -1;
}

// Bit j: row t * k + j0 + j is named by no slot (its zeros fall to this token).
__device__ __forceinline__ uint32_t unnamed_rows(const RowsArgs& a, int t, int j0) {
  int id[kSlots];
  slot_entries(a.sorted_ids, a, t, j0, id);
  uint32_t bits = 0;
#pragma unroll
  for (int j = 0; j < kSlots; ++j) bits |= j0 + j < a.k && id[j] < 0 ? 1u << j : 0u;
  return bits;
}

// Unit c of the rows that unnamed_rows found.
template <typename Row, typename Un>
__device__ __forceinline__ void zero_unit(const RowsArgs& a, int t, int j0, uint32_t bits, int c) {
#pragma unroll
  for (int j = 0; j < kSlots; ++j)
    if ((bits >> j) & 1)
      row_at<Row, typename Un::raw>(a.dst, (int64_t)t * a.k + j0 + j, a.dst_ld)[c] = Un::zero();
}

template <typename Row, bool WIDE, int G>
__global__ void __launch_bounds__(256) dispatch_kernel(const void* src, int64_t src_ld, const int32_t* slot_rows,
                                                       const int32_t* sorted_ids, int32_t n_tokens,
                                                       int32_t k, RowsArgs a) {
  a.src = src;
  a.src_ld = src_ld;
  a.slot_rows = slot_rows;
  a.sorted_ids = sorted_ids;
  a.n_tokens = n_tokens;
  a.k = k;
  typedef Unit<Row, WIDE> Un;
  typedef typename Un::raw raw;
  const int t = uniform_i32(flat_group() * (256 / G) + (int)(threadIdx.x / G));
  const int g = threadIdx.x & (G - 1);
  if (t >= a.n_tokens) return;
  const raw* x = row_at<Row, raw>(a.src, t, a.src_ld);
  for (int j0 = 0; j0 < a.k; j0 += kSlots) {
    // x is requested ahead of the row numbers, a unit ahead of its stores
    raw next = x[min(g, a.units - 1)];
    int row[kSlots];
    slot_numbers(a, t, j0, row);
    const uint32_t unnamed = unnamed_rows(a, t, j0);
    for (int c = g; c < a.units; c += G) {
      const raw v = next;
      if (c + G < a.units) next = x[c + G];
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (row[j] >= 0) store_once(&row_at<Row, raw>(a.dst, row[j], a.dst_ld)[c], v);
      if (unnamed) zero_unit<Row, Un>(a, t, j0, unnamed, c);
    }
  }
}

template <typename Row, bool WIDE, int G>
__global__ void __launch_bounds__(256) combine_kernel(const void* src, int64_t src_ld, const int32_t* slot_rows,
                                                      const float* weights, int32_t n_tokens,
                                                      int32_t k, RowsArgs a) {
  a.src = src;
  a.src_ld = src_ld;
  a.slot_rows = slot_rows;
  a.weights = weights;
  a.n_tokens = n_tokens;
  a.k = k;
  typedef Unit<Row, WIDE> Un;
  typedef typename Un::raw raw;
  const int t = uniform_i32(flat_group() * (256 / G) + (int)(threadIdx.x / G));
  const int g = threadIdx.x & (G - 1);
  if (t >= a.n_tokens) return;
  raw* out = row_at<Row, raw>(a.dst, t, a.dst_ld);
  for (int c = g; c < a.units; c += G) {
    float acc[Un::kN] = {};
    for (int j0 = 0; j0 < a.k; j0 += kSlots) {
      int row[kSlots];
      slot_numbers(a, t, j0, row);
      raw v[kSlots];
      float ws[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        v[j] = row[j] >= 0 ? load_once(&row_at<Row, raw>(a.src, row[j], a.src_ld)[c]) : Un::zero();
        ws[j] = a.weights ? a.weights[(int64_t)t * a.k + min(j0 + j, a.k - 1)] : 1.f;
      }
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        if (row[j] < 0) continue;
        const float w = ws[j];
        float f[Un::kN];
        Un::widen(v[j], f);
#pragma unroll
        for (int i = 0; i < Un::kN; ++i) acc[i] = fmaf(w, f[i], acc[i]);
      }
    }
    out[c] = Un::narrow(acc);
  }
}

template <typename Row, bool WIDE, int G>
__global__ void __launch_bounds__(256) combine_backward_kernel(const void* d_out, const int32_t* slot_rows,
                                                               const int32_t* sorted_ids,
                                                               const float* weights, int32_t n_tokens,
                                                               int32_t k, RowsArgs a) {
  a.d_out = d_out;
  a.slot_rows = slot_rows;
  a.sorted_ids = sorted_ids;
  a.weights = weights;
  a.n_tokens = n_tokens;
  a.k = k;
  typedef Unit<Row, WIDE> Un;
  typedef typename Un::raw raw;
  __shared__ float part[256 / 64][kSlots];
  // every thread of a workgroup reaches the barriers: a token past the end
  // has no slots and no columns
  const int tok = uniform_i32(flat_group() * (256 / G) + (int)(threadIdx.x / G));
  const int g = threadIdx.x & (G - 1);
  const bool on = tok < a.n_tokens;
  const int t = on ? tok : 0;
  const int units = on ? a.units : 0;
  const raw* dout = row_at<Row, raw>(a.d_out, t, a.d_out_ld);
  for (int j0 = 0; j0 < a.k; j0 += kSlots) {
    int row[kSlots];
    float w[kSlots], dot[kSlots] = {};
    slot_numbers(a, t, j0, row);
    const uint32_t unnamed = a.sorted_ids ? unnamed_rows(a, t, j0) : 0u;
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      w[j] = a.weights ? a.weights[(int64_t)t * a.k + min(j0 + j, a.k - 1)] : 1.f;
    for (int c = g; c < units; c += G) {
      float d[Un::kN];
      Un::widen(dout[c], d);
      raw v[kSlots];
      if (a.d_weights) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          v[j] = row[j] >= 0 ? load_once(&row_at<Row, raw>(a.src, row[j], a.src_ld)[c]) : Un::zero();
      }
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        if (row[j] < 0) continue;
        float o[Un::kN];
#pragma unroll
        for (int i = 0; i < Un::kN; ++i) o[i] = w[j] * d[i];
        store_once(&row_at<Row, raw>(a.dst, row[j], a.dst_ld)[c], Un::narrow(o));
        if (a.d_weights) {
          float f[Un::kN];
          Un::widen(v[j], f);
#pragma unroll
          for (int i = 0; i < Un::kN; ++i) dot[j] = fmaf(d[i], f[i], dot[j]);
        }
      }
      if (unnamed) zero_unit<Row, Un>(a, t, j0, unnamed, c);
    }
    if (a.d_weights) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j) dot[j] = group_sum<64>(dot[j]);
      const int wave = threadIdx.x >> 6;
      if constexpr (G > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
          for (int j = 0; j < kSlots; ++j) part[wave][j] = dot[j];
        }
        __syncthreads();
        if (on && g < kSlots && j0 + g < a.k) {
          float s = 0.f;
          for (int i = 0; i < G / 64; ++i) s += part[wave + i][g];
          a.d_weights[(int64_t)t * a.k + j0 + g] = s;
        }
      } else if (on) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (g == j && j0 + j < a.k) a.d_weights[(int64_t)t * a.k + j0 + j] = dot[j];
      }
    }
  }
}

enum RowsOp { kDispatch, kCombine, kCombineBackward };

template <typename Row, bool WIDE, int G>
void launch_rows(RowsOp op, const RowsArgs& a, hipStream_t s) {
  const dim3 grid = flat_grid(((int64_t)a.n_tokens * G + 255) / 256), block(256);
  if (op == kDispatch)
    hipLaunchKernelGGL((dispatch_kernel<Row, WIDE, G>), grid, block, 0, s, a.src, a.src_ld,
                       a.slot_rows, a.sorted_ids, a.n_tokens, a.k, a);
  else if (op == kCombine)
    hipLaunchKernelGGL((combine_kernel<Row, WIDE, G>), grid, block, 0, s, a.src, a.src_ld,
                       a.slot_rows, a.weights, a.n_tokens, a.k, a);
  else
    hipLaunchKernelGGL((combine_backward_kernel<Row, WIDE, G>), grid, block, 0, s, a.d_out,
                       a.slot_rows, a.sorted_ids, a.weights, a.n_tokens, a.k, a);
}

template <typename Row, bool WIDE>
void launch_rows_g(RowsOp op, const RowsArgs& a, hipStream_t s) {
  if (a.units <= 64) return launch_rows<Row, WIDE, 64>(op, a, s);
  if (a.units <= 128) return launch_rows<Row, WIDE, 128>(op, a, s);
  launch_rows<Row, WIDE, 256>(op, a, s);
}

// Units of 16 bytes where every row starts on 16 bytes and holds whole ones.
int32_t run_rows(RowsOp op, RowsArgs a, int64_t dim, int32_t dtype, const char* who,
                 hipStream_t s) {
  const int v = dtype == MLORA_BF16 ? 8 : 4;
  const bool wide = dim % v == 0 && a.src_ld % v == 0 && a.dst_ld % v == 0 &&
                    a.d_out_ld % v == 0 && aligned(a.src, 16) && aligned(a.dst, 16) &&
                    aligned(a.d_out, 16);
  a.units = (int32_t)(wide ? dim / v : dim);
  (void)hipGetLastError();
  if (dtype == MLORA_BF16) {
    if (wide)
      launch_rows_g<Bf16Row, true>(op, a, s);
    else
      launch_rows_g<Bf16Row, false>(op, a, s);
  } else {
    if (wide)
      launch_rows_g<F32Row, true>(op, a, s);
    else
      launch_rows_g<F32Row, false>(op, a, s);
  }
  return launch_status(who);
}

int32_t check_rows(const char* who, int32_t dtype, int64_t n_tokens, int64_t dim, int32_t top_k) {
  if (dtype != MLORA_BF16 && dtype != MLORA_F32)
    return fail(MLORA_ERR_INVALID, "%s: dtype %d is neither bf16 nor f32", who, dtype);
  if (top_k < 1 || top_k > kMaxTopK)
    return fail(MLORA_ERR_INVALID, "%s: top_k=%d outside [1, %d]", who, top_k, kMaxTopK);
  if (n_tokens < 0 || n_tokens > kMaxRows / top_k)
    return fail(MLORA_ERR_INVALID, "%s: n_tokens=%lld with top_k=%d out of range", who,
                (long long)n_tokens, top_k);
  if (dim < 1 || dim > kMaxRows)
    return fail(MLORA_ERR_INVALID, "%s: dim=%lld out of range", who, (long long)dim);
  return MLORA_OK;
}

int32_t check_ld(const char* who, const char* what, int64_t ld, int64_t dim) {
  if (ld < dim)
    return fail(MLORA_ERR_INVALID, "%s: row stride %lld of %s below its width %lld", who,
                (long long)ld, what, (long long)dim);
  return MLORA_OK;
}

}  // namespace
}  // namespace mlora

using namespace mlora;

extern "C" int32_t mlora_router_topk(const void* logits, int64_t logits_ld, int32_t dtype,
                                     int64_t n_tokens, int32_t n_experts, int32_t top_k,
                                     int32_t renormalize, int32_t* indices, float* weights,
                                     void* stream) {
  const char* who = "mlora_router_topk";
  if (int32_t rc = check_router(who, dtype, n_tokens, n_experts, top_k, logits_ld)) return rc;
  if (n_tokens == 0) {
    clear_error();
    return MLORA_OK;
  }
  if (!logits || !indices || !weights)
    return fail(MLORA_ERR_INVALID, "%s: NULL device pointer", who);
  RouterArgs a{};
  a.logits = logits;
  a.ld = logits_ld;
  a.indices = indices;
  a.weights = weights;
  a.n_tokens = (int32_t)n_tokens;
  a.E = n_experts;
  a.k = top_k;
  a.renorm = renormalize != 0;
  return run_router(a, dtype, false, who, reinterpret_cast<hipStream_t>(stream));
}

extern "C" int32_t mlora_router_topk_backward(const void* logits, int64_t logits_ld,
                                              int32_t dtype, int64_t n_tokens, int32_t n_experts,
                                              int32_t top_k, int32_t renormalize,
                                              const int32_t* indices, const float* d_weights,
                                              void* d_logits, int64_t d_logits_ld, void* stream) {
  const char* who = "mlora_router_topk_backward";
  if (int32_t rc = check_router(who, dtype, n_tokens, n_experts, top_k, logits_ld)) return rc;
  if (int32_t rc = check_ld(who, "d_logits", d_logits_ld, n_experts)) return rc;
  if (n_tokens == 0) {
    clear_error();
    return MLORA_OK;
  }
  if (!logits || !indices || !d_weights || !d_logits)
    return fail(MLORA_ERR_INVALID, "%s: NULL device pointer", who);
  RouterArgs a{};
  a.logits = logits;
  a.ld = logits_ld;
  a.indices = const_cast<int32_t*>(indices);
  a.d_weights = d_weights;
  a.d_logits = d_logits;
  a.d_ld = d_logits_ld;
  a.n_tokens = (int32_t)n_tokens;
  a.E = n_experts;
  a.k = top_k;
  a.renorm = renormalize != 0;
  return run_router(a, dtype, true, who, reinterpret_cast<hipStream_t>(stream));
}

extern "C" uint64_t mlora_moe_sort_workspace_bytes(int64_t n_slots, int32_t n_experts) {
  if (n_slots <= 0 || n_slots > kMaxRows || n_experts < 1 || n_experts > kMaxExperts) return 0;
  const int blocks = sort_blocks(n_slots);
  return blocks == 0 ? 0 : (((uint64_t)blocks * (n_experts + 1) * 4 + 255) & ~255ull);
}

extern "C" int32_t mlora_moe_sort(const int32_t* ids, int64_t n_slots, int32_t n_experts,
                                  int32_t* expert_offsets, int32_t* sorted_ids,
                                  int32_t* slot_rows, void* workspace, uint64_t workspace_bytes,
                                  void* stream) {
  const char* who = "mlora_moe_sort";
  if (n_slots < 0 || n_slots > kMaxRows)
    return fail(MLORA_ERR_INVALID, "%s: n_slots=%lld out of range", who, (long long)n_slots);
  if (n_experts < 1 || n_experts > kMaxExperts)
    return fail(MLORA_ERR_INVALID, "%s: n_experts=%d outside [1, %d]", who, n_experts,
                kMaxExperts);
  if (!expert_offsets || (n_slots > 0 && (!ids || !sorted_ids || !slot_rows)))
    return fail(MLORA_ERR_INVALID, "%s: NULL device pointer", who);
  if (!workspace && workspace_bytes != 0)
    return fail(MLORA_ERR_INVALID, "%s: NULL workspace with workspace_bytes > 0", who);
  if (!aligned(ids, 4))
    return fail(MLORA_ERR_INVALID, "%s: ids must be 4-byte aligned", who);
  if (!aligned(workspace, 4))
    return fail(MLORA_ERR_INVALID, "%s: workspace must be 4-byte aligned", who);
  const uint64_t need = mlora_moe_sort_workspace_bytes(n_slots, n_experts);
  if (workspace_bytes < need)
    return fail(MLORA_ERR_CAPACITY, "%s: workspace of %llu bytes, %llu needed", who,
                (unsigned long long)workspace_bytes, (unsigned long long)need);
  SortArgs a{};
  a.ids = ids;
  a.offsets = expert_offsets;
  a.sorted_ids = sorted_ids;
  a.slot_rows = slot_rows;
  a.counts = static_cast<int32_t*>(workspace);
  a.n = (int32_t)n_slots;
  a.E = n_experts;
  a.key_bits = 32 - __builtin_clz((unsigned)n_experts + 1);  // keys 0 .. E + 1
  a.tiles_per_block = 1;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const size_t lds = sort_lds_bytes(n_experts);
  const dim3 threads(kSortThreads);
  if (n_slots == 0) {
    // nothing to place: the offsets alone, all 0
    hipLaunchKernelGGL(sort_empty_kernel, dim3(1), dim3(256), 0, s, a);
  } else if (n_slots <= kSortThreads) {
    hipLaunchKernelGGL((sort_place_kernel<1, kSortAlone>), dim3(1), threads, lds, s, a.ids, a.n,
                       a.E, a.key_bits, a);
  } else if (n_slots <= kSortOne) {
    const int blocks = (int)((n_slots + kSortThreads - 1) / kSortThreads);
    const size_t counters = (size_t)2 * kSortCopies * (n_experts + 1) * 4;
    hipLaunchKernelGGL((sort_place_kernel<1, kSortRecount>), dim3(blocks), threads,
                       counters > lds ? counters : lds, s, a.ids, a.n, a.E, a.key_bits, a);
  } else {
    a.blocks = sort_blocks(n_slots);
    const int64_t tiles = (n_slots + kSortTile - 1) / kSortTile;
    a.tiles_per_block = (int32_t)((tiles + a.blocks - 1) / a.blocks);
    hipLaunchKernelGGL(sort_count_kernel, dim3(a.blocks), threads, (size_t)(n_experts + 1) * 4, s,
                       a);
    if (int32_t rc = launch_status(who)) return rc;
    hipLaunchKernelGGL((sort_place_kernel<kSortR, kSortCounted>), dim3(a.blocks), threads, lds, s,
                       a.ids, a.n, a.E, a.key_bits, a);
  }
  return launch_status(who);
}

extern "C" int32_t mlora_moe_dispatch(const void* x, int64_t x_ld, int32_t dtype,
                                      int64_t n_tokens, int64_t dim, int32_t top_k,
                                      const int32_t* sorted_ids, const int32_t* slot_rows,
                                      void* rows, int64_t rows_ld, void* stream) {
  const char* who = "mlora_moe_dispatch";
  if (int32_t rc = check_rows(who, dtype, n_tokens, dim, top_k)) return rc;
  if (int32_t rc = check_ld(who, "x", x_ld, dim)) return rc;
  if (int32_t rc = check_ld(who, "rows", rows_ld, dim)) return rc;
  if (n_tokens == 0) {
    clear_error();
    return MLORA_OK;
  }
  if (!x || !sorted_ids || !slot_rows || !rows)
    return fail(MLORA_ERR_INVALID, "%s: NULL device pointer", who);
  RowsArgs a{};
  a.src = x;
  a.src_ld = x_ld;
  a.dst = rows;
  a.dst_ld = rows_ld;
  a.slot_rows = slot_rows;
  a.sorted_ids = sorted_ids;
  a.n_rows = n_tokens * top_k;
  a.n_tokens = (int32_t)n_tokens;
  a.k = top_k;
  return run_rows(kDispatch, a, dim, dtype, who, reinterpret_cast<hipStream_t>(stream));
}

extern "C" int32_t mlora_moe_combine(const void* rows, int64_t rows_ld, int64_t n_rows,
                                     int32_t dtype, int64_t n_tokens, int64_t dim, int32_t top_k,
                                     const float* weights, const int32_t* slot_rows, void* out,
                                     int64_t out_ld, void* stream) {
  const char* who = "mlora_moe_combine";
  if (int32_t rc = check_rows(who, dtype, n_tokens, dim, top_k)) return rc;
  if (int32_t rc = check_ld(who, "rows", rows_ld, dim)) return rc;
  if (int32_t rc = check_ld(who, "out", out_ld, dim)) return rc;
  if (n_rows < 0 || n_rows > kMaxRows || (!slot_rows && n_rows < n_tokens * top_k))
    return fail(MLORA_ERR_INVALID, "%s: n_rows=%lld out of range", who, (long long)n_rows);
  if (n_tokens == 0) {
    clear_error();
    return MLORA_OK;
  }
  if ((n_rows > 0 && !rows) || !out)
    return fail(MLORA_ERR_INVALID, "%s: NULL device pointer", who);
  RowsArgs a{};
  a.src = rows;
  a.src_ld = rows_ld;
  a.dst = out;
  a.dst_ld = out_ld;
  a.weights = weights;
  a.slot_rows = slot_rows;
  a.n_rows = n_rows;
  a.n_tokens = (int32_t)n_tokens;
  a.k = top_k;
  return run_rows(kCombine, a, dim, dtype, who, reinterpret_cast<hipStream_t>(stream));
}

extern "C" int32_t mlora_moe_combine_backward(const void* d_out, int64_t d_out_ld,
                                              const void* rows, int64_t rows_ld, int32_t dtype,
                                              int64_t n_tokens, int64_t dim, int32_t top_k,
                                              const float* weights, const int32_t* slot_rows,
                                              const int32_t* sorted_ids, void* d_rows,
                                              int64_t d_rows_ld, float* d_weights, void* stream) {
  const char* who = "mlora_moe_combine_backward";
  if (int32_t rc = check_rows(who, dtype, n_tokens, dim, top_k)) return rc;
  if (int32_t rc = check_ld(who, "d_out", d_out_ld, dim)) return rc;
  if (int32_t rc = check_ld(who, "d_rows", d_rows_ld, dim)) return rc;
  if (d_weights)
    if (int32_t rc = check_ld(who, "rows", rows_ld, dim)) return rc;
  if ((slot_rows == nullptr) != (sorted_ids == nullptr))
    return fail(MLORA_ERR_INVALID, "%s: slot_rows and sorted_ids go together", who);
  if (n_tokens == 0) {
    clear_error();
    return MLORA_OK;
  }
  if (!d_out || !d_rows || (d_weights && !rows))
    return fail(MLORA_ERR_INVALID, "%s: NULL device pointer", who);
  RowsArgs a{};
  a.src = d_weights ? rows : nullptr;
  a.src_ld = d_weights ? rows_ld : 0;
  a.d_out = d_out;
  a.d_out_ld = d_out_ld;
  a.dst = d_rows;
  a.dst_ld = d_rows_ld;
  a.weights = weights;
  a.slot_rows = slot_rows;
  a.sorted_ids = sorted_ids;
  a.d_weights = d_weights;
  a.n_rows = n_tokens * top_k;
  a.n_tokens = (int32_t)n_tokens;
  a.k = top_k;
  return run_rows(kCombineBackward, a, dim, dtype, who, reinterpret_cast<hipStream_t>(stream));
}
