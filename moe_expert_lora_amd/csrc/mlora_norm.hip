// The norms before and after a block, with its gate and residual scale, and
// their gradients, for gfx950 (MI355X).
#include <algorithm>
#include <cmath>

#include "mlora_device.h"

namespace mlora {
namespace {

// Of each row, with R(v) = 1 / sqrt(mean(v^2) + eps):
//   n = y R(y) (wy + offset)   (no wy: n = y)
//   r = residual_scale residual + y_scale gate n
//   x = r R(r) (wx + offset)
// One pass: a row's values stay in registers from the first load to the last
// store, as fp32; r enters the second norm unrounded. 64 to 1024 threads
// hold a row, 8 or 16 values each, and keep the weights from row to row; the two
// means are sums over them in a fixed order. The gradients recompute r from the
// same inputs (which are read for the norms' gradients anyway), so nothing is
// saved forward:
//   g = d_x (wx + offset), h = r R(r)
//   d = d_r + R(r) (g - h mean(g h))              the gradient of r
//   d_residual = residual_scale d, d_gate = y_scale d n, d_n = y_scale d gate
//   d_y = R(y) (u - v mean(u v)), u = d_n (wy + offset), v = y R(y)
// Gradients of what all rows share (wx, wy, a gate per channel) are summed over a
// thread's rows in registers and over a workgroup's rows in LDS, written once per
// workgroup, and added up by a second kernel in a fixed order.

enum GateForm { kNoGate, kChannel, kToken, kFull };
constexpr int kMaxDim = 16384;
constexpr int kSums = 3;          // wx, wy, gate per channel

struct NormArgs {
  mlora_norm_block b;
  void* r;
  int64_t r_ld;
  void* x;
  int64_t x_ld;
  const void *d_r, *d_x;  // gradients from here on
  int64_t d_r_ld, d_x_ld;
  void *d_residual, *d_y, *d_gate;
  int64_t d_residual_ld, d_y_ld, d_gate_ld;
  float* partial[kSums];  // [workgroups][dim], null: not wanted
  bool past;              // the outputs are too large to be found in a cache later
};

// A thread's VPT values of a row: neighbours that fill 16 bytes, threads in turn.
template <typename Row, int TPR, int VPT>
struct Cols {
  typedef typename Row::elem elem;
  static constexpr int V = Row::kPer16;
  static constexpr int CH = VPT / V;
  // More than 512 values a row (shape_of): no code for rows of less than a vector. Not of
  // 1024 threads, whose few registers happen to be spilled worse without it (gradients of
  // 2000 rows of 16384: 474 -> 630 us).
  static constexpr bool kWide = TPR > 64 && TPR < 1024;
  static __device__ __forceinline__ int col(int ch, int tid) { return (ch * TPR + tid) * V; }

  // A row as it is loaded, so that the next row's loads can be on their way.
  struct Raw {
    u32x4 v[CH];
  };
  static __device__ __forceinline__ void request(const void* base, int64_t off, int D, int tid,
                                                 Raw& r) {
    const elem* p = static_cast<const elem*>(base) + off;
    if (kWide || D >= V) {
#pragma unroll
      for (int c = 0; c < CH; ++c) r.v[c] = load16_row<Row, false, true>(p, col(c, tid), D);
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) r.v[c] = load16_row<Row, true>(p, col(c, tid), D);
    }
  }
  static __device__ __forceinline__ void widen(const Raw& r, int D, int tid, float (&f)[VPT]) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      Row::widen16(row16_tail<Row, kWide>(r.v[c], col(c, tid), D), f + c * V);
  }
  // past: past the caches' keep
  static __device__ __forceinline__ void store(void* base, int64_t off, int D, int tid,
                                               const float (&f)[VPT], bool past) {
    elem* p = static_cast<elem*>(base) + off;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (col(c, tid) >= D) continue;
      const u32x4 v = Row::narrow16(f + c * V);
      if (past)
        store16_any<Row, true>(p + col(c, tid), D - col(c, tid), v);
      else
        store16_any<Row>(p + col(c, tid), D - col(c, tid), v);
    }
  }
  // fp32 vectors of the row's width
  static __device__ __forceinline__ void store_f32(float* p, int D, int tid, const float (&f)[VPT]) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < V; i += 4)
        if (col(c, tid) + i < D)
          store16_any<F32Row>(p + col(c, tid) + i, D - col(c, tid) - i,
                              F32Row::narrow16(f + c * V + i));
  }
  // norm weights plus offset, of either type; null: 1. Zeros past the row.
  template <typename W>
  static __device__ __forceinline__ void load_weight_as(const void* w, float offset, int D, int tid,
                                                        float (&f)[VPT]) {
    const typename W::elem* p = static_cast<const typename W::elem*>(w);
    auto load = [&](const typename W::elem* p, int at) {
      return kWide || D >= W::kPer16 ? row16_tail<W, kWide>(load16_row<W, false>(p, at, D), at, D)
                            : load16_row<W, true>(p, at, D);
    };
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float g[V < W::kPer16 ? W::kPer16 : V];
#pragma unroll
      for (int i = 0; i < V; i += W::kPer16)
        W::widen16(load(p, col(c, tid) + i), g + i);
#pragma unroll
      for (int i = 0; i < V; ++i) f[c * V + i] = col(c, tid) + i < D ? g[i] + offset : 0.f;
    }
  }
  static __device__ __forceinline__ void load_weight(const void* w, int dtype, float offset, int D,
                                                     int tid, float (&f)[VPT]) {
    if (!w) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) f[i] = col(i / V, tid) + i % V < D ? 1.f : 0.f;
    } else if (dtype == MLORA_F32) {
      load_weight_as<F32Row>(w, offset, D, tid, f);
    } else {
      load_weight_as<Bf16Row>(w, offset, D, tid, f);
    }
  }
};

// N sums over a row's threads, the same in all of them. `lds`: N * TPR / 64
// floats that no earlier sum of the row still reads.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* lds, int tid) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = group_sum<64>(v[i]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    if ((tid & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) lds[i * W + (tid >> 6)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[i] += lds[i * W + w];
    }
  }
}

__device__ __forceinline__ float inv_rms(float sum, int D, float eps) {
  return 1.f / sqrtf(sum / (float)D + eps);
}

// y -> v = y R(y) and n, R(y); n = y where there is no wy.
template <typename C, int TPR, int VPT>
__device__ __forceinline__ float norm_y(const mlora_norm_block& b, const float (&y)[VPT],
                                        const float (&wy)[VPT], float* lds, int tid, float (&n)[VPT]) {
  if (!b.y_weight) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) n[i] = y[i];
    return 1.f;
  }
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) s[0] += y[i] * y[i];
  row_sums<TPR, 1>(s, lds, tid);
  const float R = inv_rms(s[0], b.dim, b.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) n[i] = y[i] * R * wy[i];
  return R;
}

// Threads of a workgroup: one row's, or four waves with a row each.
constexpr int threads_of(int tpr) { return tpr < 128 ? 256 : tpr; }
constexpr int rows_of(int tpr) { return threads_of(tpr) / tpr; }

// What a row's loads bring.
template <typename C>
struct RowIn {
  typename C::Raw residual, y, gate, d_r, d_x;
  float token_gate;
};
template <typename Row, typename C>
__device__ __forceinline__ void request_row(const NormArgs& a, int64_t row, int tid, RowIn<C>& in) {
  const mlora_norm_block& b = a.b;
  C::request(b.residual, row * b.residual_ld, b.dim, tid, in.residual);
  if (b.y) C::request(b.y, row * b.y_ld, b.dim, tid, in.y);
  if (b.gate_form == kFull) C::request(b.gate, row * b.gate_ld, b.dim, tid, in.gate);
  in.token_gate = 1.f;
  if (b.gate_form == kToken)
    in.token_gate = Row::widen(static_cast<const typename Row::elem*>(b.gate)[row * b.gate_ld]);
}
template <typename C>
__device__ __forceinline__ void request_gradients(const NormArgs& a, int64_t row, int tid,
                                                  RowIn<C>& in) {
  const mlora_norm_block& b = a.b;
  if (a.d_r) C::request(a.d_r, row * a.d_r_ld, b.dim, tid, in.d_r);
  if (a.d_x) C::request(a.d_x, row * a.d_x_ld, b.dim, tid, in.d_x);
}
// The gate of each of the thread's values; a gate per channel is in in.gate already.
template <typename C, int VPT>
__device__ __forceinline__ void gate_of(const mlora_norm_block& b, const RowIn<C>& in, int tid,
                                        float (&f)[VPT]) {
  if (b.gate_form == kFull || b.gate_form == kChannel) {
    C::widen(in.gate, b.dim, tid, f);
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) f[i] = in.token_gate;
  }
}

template <typename Row, int TPR, int VPT>
__global__ void __launch_bounds__(threads_of(TPR)) norm_forward_kernel(NormArgs a) {
  typedef Cols<Row, TPR, VPT> C;
  // of alternate rows: a wave may write the next row's sums while another reads
  __shared__ float sums[2][2][TPR / 64];
  const mlora_norm_block& b = a.b;
  const int tid = threadIdx.x & (TPR - 1), D = b.dim;
  const int64_t groups = (int64_t)gridDim.x * rows_of(TPR);
  float wx[VPT], wy[VPT];
  RowIn<C> in;
  if (a.x) C::load_weight(b.x_weight, b.w_dtype, b.weight_offset, D, tid, wx);
  if (b.y_weight) C::load_weight(b.y_weight, b.w_dtype, b.weight_offset, D, tid, wy);
  if (b.gate_form == kChannel) C::request(b.gate, 0, D, tid, in.gate);
  int odd = 0;
  // all of a row's threads (one wave, or the workgroup) leave together
  for (int64_t row = (int64_t)blockIdx.x * rows_of(TPR) + threadIdx.x / TPR; row < b.n_tokens;
       row += groups, odd ^= 1) {
    request_row<Row, C>(a, row, tid, in);
    float r[VPT];
    C::widen(in.residual, b.dim, tid, r);
    if (b.y) {
      float y[VPT], gate[VPT], n[VPT];
      C::widen(in.y, b.dim, tid, y);
      gate_of<C, VPT>(b, in, tid, gate);
      norm_y<C, TPR, VPT>(b, y, wy, sums[odd][0], tid, n);
#pragma unroll
      for (int i = 0; i < VPT; ++i) r[i] = b.residual_scale * r[i] + b.y_scale * gate[i] * n[i];
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) r[i] *= b.residual_scale;
    }
    if (a.r) C::store(a.r, row * a.r_ld, D, tid, r, a.past);
    if (!a.x) continue;  // of the whole call
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) s[0] += r[i] * r[i];
    row_sums<TPR, 1>(s, sums[odd][1], tid);
    const float R = inv_rms(s[0], D, b.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) r[i] *= R * wx[i];
    C::store(a.x, row * a.x_ld, D, tid, r, a.past);
  }
}

template <typename Row, int TPR, int VPT>
__global__ void __launch_bounds__(threads_of(TPR)) norm_backward_kernel(NormArgs a) {
  typedef Cols<Row, TPR, VPT> C;
  __shared__ float sums[2][5][TPR / 64];  // of alternate rows
  const mlora_norm_block& b = a.b;
  const int tid = threadIdx.x & (TPR - 1), D = b.dim;
  const int64_t group = (int64_t)blockIdx.x * rows_of(TPR) + threadIdx.x / TPR;
  const int64_t groups = (int64_t)gridDim.x * rows_of(TPR);
  float wx[VPT], wy[VPT], sum_wx[VPT], sum_wy[VPT], sum_gate[VPT];
  C::load_weight(b.x_weight, b.w_dtype, b.weight_offset, D, tid, wx);
  if (b.y_weight) C::load_weight(b.y_weight, b.w_dtype, b.weight_offset, D, tid, wy);
#pragma unroll
  for (int i = 0; i < VPT; ++i) sum_wx[i] = sum_wy[i] = sum_gate[i] = 0.f;

  RowIn<C> in;
  if (b.gate_form == kChannel) C::request(b.gate, 0, D, tid, in.gate);
  // 8 values a thread leave registers for the next row's loads; 16 do not, nor for the
  // gradients before they are needed (2000 rows of 8192 85 -> 74 us)
  constexpr bool kAhead = VPT <= 8;
  if (kAhead && group < b.n_tokens) {
    request_row<Row, C>(a, group, tid, in);
    request_gradients<C>(a, group, tid, in);
  }
  int odd = 0;
  for (int64_t row = group; row < b.n_tokens; row += groups, odd ^= 1) {
    float(*lds)[TPR / 64] = sums[odd];
    if (!kAhead) request_row<Row, C>(a, row, tid, in);
    float r[VPT], y[VPT], d[VPT], g[VPT], gate[VPT], n[VPT];
    C::widen(in.residual, b.dim, tid, r);
    float Ry = 1.f;
    if (b.y) {
      C::widen(in.y, b.dim, tid, y);
      gate_of<C, VPT>(b, in, tid, gate);
    }
    auto take_gradients = [&] {
      if (a.d_r) {
        C::widen(in.d_r, b.dim, tid, d);
      } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) d[i] = 0.f;
      }
      if (a.d_x) C::widen(in.d_x, b.dim, tid, g);
    };
    if (kAhead) take_gradients();
    // the next row's loads are on their way through this row's sums
    if (kAhead && row + groups < b.n_tokens) {
      request_row<Row, C>(a, row + groups, tid, in);
      request_gradients<C>(a, row + groups, tid, in);
    }
    if (b.y) {
      Ry = norm_y<C, TPR, VPT>(b, y, wy, lds[0], tid, n);
#pragma unroll
      for (int i = 0; i < VPT; ++i) r[i] = b.residual_scale * r[i] + b.y_scale * gate[i] * n[i];
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) r[i] *= b.residual_scale;
    }
    if (!kAhead) {
      request_gradients<C>(a, row, tid, in);
      take_gradients();
    }
    if (a.d_x) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        s[0] += r[i] * r[i];
        s[1] += g[i] * wx[i] * r[i];
      }
      row_sums<TPR, 2>(s, lds[1], tid);
      const float R = inv_rms(s[0], D, b.eps);
      const float mean = s[1] * R / (float)D;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const float h = r[i] * R;
        sum_wx[i] += g[i] * h;
        d[i] += R * (g[i] * wx[i] - h * mean);
      }
    }
    if (a.d_residual) {
      float out[VPT];
#pragma unroll
      for (int i = 0; i < VPT; ++i) out[i] = b.residual_scale * d[i];
      C::store(a.d_residual, row * a.d_residual_ld, D, tid, out, a.past);
    }
    if (!b.y) continue;  // of the whole call
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      d[i] *= b.y_scale;
      const float dg = d[i] * n[i];  // of the gate
      n[i] = dg;
      sum_gate[i] += dg;
      s[0] += dg;
      d[i] *= gate[i];  // of n
      if (b.y_weight) {
        y[i] *= Ry;
        sum_wy[i] += d[i] * y[i];
        d[i] *= wy[i];
        s[1] += d[i] * y[i];
      }
    }
    if (b.y_weight || b.gate_form == kToken) {
      row_sums<TPR, 2>(s, lds[3], tid);
      if (b.y_weight) {
        const float mean = s[1] / (float)D;
#pragma unroll
        for (int i = 0; i < VPT; ++i) d[i] = Ry * (d[i] - y[i] * mean);
      }
    }
    if (a.d_y) C::store(a.d_y, row * a.d_y_ld, D, tid, d, a.past);
    if (a.d_gate && b.gate_form == kToken && tid == 0)
      static_cast<float*>(a.d_gate)[row * a.d_gate_ld] = s[0];
    if (a.d_gate && b.gate_form == kFull) C::store(a.d_gate, row * a.d_gate_ld, D, tid, n, a.past);
  }
  auto write_sum = [&](int which, float(&sum)[VPT]) {
    if (!a.partial[which]) return;  // of the whole call
    if constexpr (rows_of(TPR) > 1) {  // the workgroup's rows together, in their order
      __shared__ float others[rows_of(TPR) - 1][VPT][TPR];
      const int wave = threadIdx.x / TPR;
      if (wave > 0) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) others[wave - 1][i][tid] = sum[i];
      }
      __syncthreads();
      if (wave == 0) {
#pragma unroll
        for (int w = 0; w < rows_of(TPR) - 1; ++w)
#pragma unroll
          for (int i = 0; i < VPT; ++i) sum[i] += others[w][i][tid];
      }
      __syncthreads();
      if (wave > 0) return;
    }
    C::store_f32(a.partial[which] + (int64_t)blockIdx.x * D, D, tid, sum);
  };
  write_sum(0, sum_wx);
  write_sum(1, sum_wy);
  write_sum(2, sum_gate);
}

// Column sums of the groups' partial sums: 32 columns a workgroup, 32 threads a
// column, four loads of each on their way.
struct SumArgs {
  const float* partial[kSums];
  float* out[kSums];
  int32_t groups, dim;
};

__global__ void __launch_bounds__(1024) norm_sum_kernel(SumArgs a) {
  __shared__ float lds[32][33];
  const int c = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  if (!a.out[blockIdx.y]) return;
  const float* p = a.partial[blockIdx.y] + col;
  float s = 0.f;
  if (col < a.dim) {
    int g = part;
    for (; g + 96 < a.groups; g += 128) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = p[(int64_t)(g + 32 * i) * a.dim];
      s += (v[0] + v[1]) + (v[2] + v[3]);
    }
    for (; g < a.groups; g += 32) s += p[(int64_t)g * a.dim];
  }
  lds[c][part] = s;
  __syncthreads();
  // column `part`'s 32 sums in the lanes of half a wave
  s = group_sum<32>(lds[part][c]);
  const int out_col = blockIdx.x * 32 + part;
  if (c == 0 && out_col < a.dim) a.out[blockIdx.y][out_col] = s;
}

// Threads per row and values per thread: 8, as far as 1024 threads go; the gradients
// hold twice as much a value, and take 16 in 512 threads rather than 8 in 1024.
struct Shape {
  int tpr, vpt;
};
Shape shape_of(int dim, bool backward) {
  if (dim <= 512) return {64, 8};
  if (dim <= 1024) return {128, 8};
  if (dim <= 2048) return {256, 8};
  if (dim <= 4096) return {512, 8};
  if (dim <= 8192) return backward ? Shape{512, 16} : Shape{1024, 8};
  return {1024, 16};
}
// Workgroups that go through n_tokens rows, at most `most`, each about as many.
int64_t grid_of(int64_t n_tokens, Shape h, int64_t most) {
  const int64_t per = rows_of(h.tpr), groups = (n_tokens + per - 1) / per;
  const int64_t turns = (groups + most - 1) / most;
  return (groups + turns - 1) / turns;
}
// Of the gradients: two waves a SIMD, since each workgroup writes sums of its own.
// One, two, four and six a SIMD measured 45, 32, 39 and 40 us (4096 rows of 2048), 46, 37,
// 45 and 45 (8000 of 300), 71, 71, 89 and 103 (2000 of 8192) when this was chosen.
int64_t backward_most(int dim) {
  const int64_t waves = 2 * 4 * 256;
  return std::max<int64_t>(256, waves * 64 / threads_of(shape_of(dim, true).tpr));
}
int64_t backward_grid(int64_t n_tokens, int dim) {
  return grid_of(n_tokens, shape_of(dim, true), backward_most(dim));
}
// What the workspace holds sums of: no fewer for more tokens, unlike the grid, whose
// even turns take fewer workgroups just past a multiple of the most.
int64_t backward_space(int64_t n_tokens, int dim) {
  const int64_t per = rows_of(shape_of(dim, true).tpr);
  return std::min((n_tokens + per - 1) / per, backward_most(dim));
}

template <typename Row, int TPR, int VPT>
void launch(const NormArgs& a, bool backward, hipStream_t s) {
  constexpr int threads = threads_of(TPR);
  const int64_t grid = backward ? backward_grid(a.b.n_tokens, a.b.dim)
                                : grid_of(a.b.n_tokens, Shape{TPR, VPT}, 256 * 2048 / threads);
  // shapes of one direction alone
  constexpr bool kForward = !(TPR == 512 && VPT == 16), kBackward = !(TPR == 1024 && VPT == 8);
  if constexpr (kBackward)
    if (backward)
      hipLaunchKernelGGL((norm_backward_kernel<Row, TPR, VPT>), dim3((unsigned)grid), dim3(threads),
                         0, s, a);
  if constexpr (kForward)
    if (!backward)
      hipLaunchKernelGGL((norm_forward_kernel<Row, TPR, VPT>), dim3((unsigned)grid), dim3(threads),
                         0, s, a);
}

template <typename Row>
void launch_shape(const NormArgs& a, bool backward, hipStream_t s) {
  const Shape h = shape_of(a.b.dim, backward);
  if (h.tpr == 64) return launch<Row, 64, 8>(a, backward, s);
  if (h.tpr == 128) return launch<Row, 128, 8>(a, backward, s);
  if (h.tpr == 256) return launch<Row, 256, 8>(a, backward, s);
  if (h.tpr == 512 && h.vpt == 8) return launch<Row, 512, 8>(a, backward, s);
  if (h.tpr == 512) return launch<Row, 512, 16>(a, backward, s);
  if (h.vpt == 8) return launch<Row, 1024, 8>(a, backward, s);
  launch<Row, 1024, 16>(a, backward, s);
}

// Rows past the size of the XCDs' L2s (8 of 4 MB) pass the caches by: 8192 rows of 4096
// bf16 values 60 -> 56 us; smaller ones may still be there for the call that reads them.
int32_t run(const char* who, NormArgs a, bool backward, hipStream_t s) {
  const mlora_norm_block& b = a.b;
  a.past = b.n_tokens * b.dim * (b.dtype == MLORA_BF16 ? 2 : 4) > (32ll << 20);
  (void)hipGetLastError();
  if (b.dtype == MLORA_BF16)
    launch_shape<Bf16Row>(a, backward, s);
  else
    launch_shape<F32Row>(a, backward, s);
  return launch_status(who);
}

int32_t check(const char* who, const mlora_norm_block* b) {
  if (!b) return fail(MLORA_ERR_INVALID, "%s: NULL block", who);
  if (b->dtype != MLORA_BF16 && b->dtype != MLORA_F32)
    return fail(MLORA_ERR_INVALID, "%s: dtype %d is neither bf16 nor f32", who, b->dtype);
  if (b->w_dtype != MLORA_BF16 && b->w_dtype != MLORA_F32)
    return fail(MLORA_ERR_INVALID, "%s: weight dtype %d is neither bf16 nor f32", who, b->w_dtype);
  if (b->n_tokens < 0 || b->n_tokens > kMaxRows)
    return fail(MLORA_ERR_INVALID, "%s: n_tokens=%lld out of range", who, (long long)b->n_tokens);
  if (b->dim < 1 || b->dim > kMaxDim)
    return fail(MLORA_ERR_INVALID, "%s: dim=%d outside [1, %d]", who, b->dim, kMaxDim);
  if (b->gate_form < kNoGate || b->gate_form > kFull)
    return fail(MLORA_ERR_INVALID, "%s: gate form %d outside [0, 3]", who, b->gate_form);
  if (!(b->eps >= 0.f) || std::isinf(b->eps))
    return fail(MLORA_ERR_INVALID, "%s: eps is negative or not finite", who);
  if (b->residual_ld < b->dim || (b->y && b->y_ld < b->dim) ||
      (b->gate_form == kFull && b->gate_ld < b->dim) ||
      (b->gate_form == kToken && b->gate_ld < 1))
    return fail(MLORA_ERR_INVALID, "%s: row stride below the row's width", who);
  if (!b->y && (b->y_weight || b->gate_form != kNoGate))
    return fail(MLORA_ERR_INVALID, "%s: a norm weight or gate for a y that is not there", who);
  if (b->n_tokens > 0 && !b->residual) return fail(MLORA_ERR_INVALID, "%s: NULL residual", who);
  if ((b->n_tokens > 0 || b->gate_form == kChannel) && (b->gate_form != kNoGate) && !b->gate)
    return fail(MLORA_ERR_INVALID, "%s: NULL gate", who);
  return MLORA_OK;
}

}  // namespace
}  // namespace mlora

using namespace mlora;

extern "C" int32_t mlora_block_norm(const mlora_norm_block* block, void* r, int64_t r_ld, void* x,
                                    int64_t x_ld, void* stream) {
  const char* who = "mlora_block_norm";
  if (int32_t rc = check(who, block)) return rc;
  if ((r && r_ld < block->dim) || (x && x_ld < block->dim))
    return fail(MLORA_ERR_INVALID, "%s: row stride below dim=%d", who, block->dim);
  if (block->n_tokens == 0) {
    clear_error();
    return MLORA_OK;
  }
  if (!r && !x) return fail(MLORA_ERR_INVALID, "%s: neither r nor x", who);
  if (r && r == x) return fail(MLORA_ERR_INVALID, "%s: r and x are the same memory", who);
  NormArgs a{};
  a.b = *block;
  a.r = r;
  a.r_ld = r_ld;
  a.x = x;
  a.x_ld = x_ld;
  return run(who, a, false, reinterpret_cast<hipStream_t>(stream));
}

extern "C" uint64_t mlora_block_norm_backward_workspace_bytes(int64_t n_tokens, int32_t dim) {
  if (n_tokens < 1 || n_tokens > kMaxRows || dim < 1 || dim > kMaxDim) return 0;
  const uint64_t groups = backward_space(n_tokens, dim);
  return (kSums * groups * dim * 4 + 255) / 256 * 256;
}

extern "C" int32_t mlora_block_norm_backward(
    const mlora_norm_block* block, const void* d_r, int64_t d_r_ld, const void* d_x, int64_t d_x_ld,
    void* d_residual, int64_t d_residual_ld, void* d_y, int64_t d_y_ld, float* d_x_weight,
    float* d_y_weight, void* d_gate, int64_t d_gate_ld, void* workspace, uint64_t workspace_bytes,
    void* stream) {
  const char* who = "mlora_block_norm_backward";
  if (int32_t rc = check(who, block)) return rc;
  const int32_t dim = block->dim;
  if ((d_r && d_r_ld < dim) || (d_x && d_x_ld < dim) || (d_residual && d_residual_ld < dim) ||
      (d_y && d_y_ld < dim) || (d_gate && block->gate_form == kFull && d_gate_ld < dim) ||
      (d_gate && block->gate_form == kToken && d_gate_ld < 1))
    return fail(MLORA_ERR_INVALID, "%s: row stride below the row's width", who);
  if (d_y && !block->y) return fail(MLORA_ERR_INVALID, "%s: d_y for a y that is not there", who);
  if (d_y_weight && !block->y_weight)
    return fail(MLORA_ERR_INVALID, "%s: d_y_weight for a y_weight that is not there", who);
  if (d_gate && block->gate_form == kNoGate)
    return fail(MLORA_ERR_INVALID, "%s: d_gate for a gate that is not there", who);
  if (block->n_tokens > 0 && !d_r && !d_x)
    return fail(MLORA_ERR_INVALID, "%s: neither d_r nor d_x", who);
  float* sums[kSums] = {d_x_weight, d_y_weight,
                        block->gate_form == kChannel ? static_cast<float*>(d_gate) : nullptr};
  const bool any = sums[0] || sums[1] || sums[2];
  NormArgs a{};
  SumArgs sa{};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (block->n_tokens > 0) {
    const uint64_t need = mlora_block_norm_backward_workspace_bytes(block->n_tokens, dim);
    if (any && (!workspace || workspace_bytes < need))
      return fail(MLORA_ERR_CAPACITY, "%s: workspace of %llu bytes, %llu needed", who,
                  (unsigned long long)(workspace ? workspace_bytes : 0), (unsigned long long)need);
    if (any && !aligned(workspace, 256))
      return fail(MLORA_ERR_INVALID, "%s: workspace must be 256-byte aligned", who);
    const void* outputs[] = {d_residual, d_y, d_x_weight, d_y_weight, d_gate};
    for (int i = 0; i < 5; ++i)
      for (int j = 0; j < i; ++j)
        if (outputs[i] && outputs[i] == outputs[j])
          return fail(MLORA_ERR_INVALID, "%s: two outputs are the same memory", who);
    a.b = *block;
    a.d_r = d_r;
    a.d_r_ld = d_r_ld;
    a.d_x = d_x;
    a.d_x_ld = d_x_ld;
    a.d_residual = d_residual;
    a.d_residual_ld = d_residual_ld;
    a.d_y = d_y;
    a.d_y_ld = d_y_ld;
    a.d_gate = d_gate;
    a.d_gate_ld = d_gate_ld;
    sa.groups = (int32_t)backward_grid(block->n_tokens, dim);
    for (int i = 0; i < kSums; ++i)
      if (sums[i])
        sa.partial[i] = a.partial[i] = static_cast<float*>(workspace) + (int64_t)i * sa.groups * dim;
    if (int32_t rc = run(who, a, true, s)) return rc;
  }
  if (any) {
    sa.dim = dim;
    for (int i = 0; i < kSums; ++i) sa.out[i] = sums[i];
    (void)hipGetLastError();
    hipLaunchKernelGGL(norm_sum_kernel, dim3((dim + 31) / 32, kSums), dim3(1024), 0, s, sa);
    return launch_status(who);
  }
  clear_error();
  return MLORA_OK;
}
