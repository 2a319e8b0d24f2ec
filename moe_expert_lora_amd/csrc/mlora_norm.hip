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
// store, as fp32; r enters the second norm unrounded. 64, 256, 512 or 1024
// threads hold a row, 8 or 16 values each; the two means are sums over them in a
// fixed order. The gradients recompute r from the same inputs (which are read
// for the norms' gradients anyway), so nothing is saved forward:
//   g = d_x (wx + offset), h = r R(r)
//   d = d_r + R(r) (g - h mean(g h))              the gradient of r
//   d_residual = residual_scale d, d_gate = y_scale d n, d_n = y_scale d gate
//   d_y = R(y) (u - v mean(u v)), u = d_n (wy + offset), v = y R(y)
// Gradients of what all rows share (wx, wy, a gate per channel) are summed over a
// thread's rows in registers, written once per group of threads, and added up by
// a second kernel in a fixed order.

enum GateForm { kNoGate, kChannel, kToken, kFull };
constexpr int kMaxDim = 16384;
constexpr int kSums = 3;          // wx, wy, gate per channel
constexpr int kMaxGroups = 1024;  // groups of threads that write partial sums

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
  float* partial[kSums];  // [groups][dim], null: not wanted
};

// A thread's VPT values of a row: neighbours that fill 16 bytes (WIDE) or single
// ones, threads in turn.
template <typename Row, int TPR, int VPT, bool WIDE>
struct Cols {
  static constexpr int V = WIDE ? Row::kPer16 : 1;
  static constexpr int CH = VPT / V;
  static __device__ __forceinline__ int col(int ch, int tid) { return (ch * TPR + tid) * V; }

  static __device__ __forceinline__ void load(const void* base, int64_t off, int D, int tid,
                                              float (&f)[VPT]) {
    const typename Row::elem* p = static_cast<const typename Row::elem*>(base) + off;
    if constexpr (WIDE) {
      u32x4 v[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        v[c] = u32x4{0, 0, 0, 0};
        if (col(c, tid) < D) v[c] = *reinterpret_cast<const u32x4*>(p + col(c, tid));
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) Row::widen16(v[c], f + c * V);
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) f[c] = col(c, tid) < D ? Row::widen(p[col(c, tid)]) : 0.f;
    }
  }
  static __device__ __forceinline__ void store(void* base, int64_t off, int D, int tid,
                                               const float (&f)[VPT]) {
    typename Row::elem* p = static_cast<typename Row::elem*>(base) + off;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (col(c, tid) >= D) continue;
      if constexpr (WIDE)
        *reinterpret_cast<u32x4*>(p + col(c, tid)) = Row::narrow16(f + c * V);
      else
        p[col(c, tid)] = Row::narrow(f[c]);
    }
  }
  // fp32 vectors of the row's width
  static __device__ __forceinline__ void store_f32(float* p, int D, int tid, const float (&f)[VPT]) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (col(c, tid) + i < D) p[col(c, tid) + i] = f[c * V + i];
  }
  // norm weights plus offset, of either type; null: 1. Zeros past the row.
  static __device__ __forceinline__ void load_weight(const void* w, int dtype, float offset, int D,
                                                     int tid, float (&f)[VPT]) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int at = col(c, tid) + i;
        float v = 0.f;
        if (at < D) {
          if (!w)
            v = 1.f;
          else if (dtype == MLORA_F32)
            v = static_cast<const float*>(w)[at] + offset;
          else
            v = Bf16Row::widen(static_cast<const uint16_t*>(w)[at]) + offset;
        }
        f[c * V + i] = v;
      }
    }
  }
  // the gate of each of the thread's values
  static __device__ __forceinline__ void load_gate(const mlora_norm_block& b, int64_t row, int tid,
                                                   float (&f)[VPT]) {
    if (b.gate_form == kFull || b.gate_form == kChannel) {
      load(b.gate, b.gate_form == kFull ? row * b.gate_ld : 0, b.dim, tid, f);
    } else {
      const float v = b.gate_form == kToken
                          ? Row::widen(static_cast<const typename Row::elem*>(b.gate)[row * b.gate_ld])
                          : 1.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) f[i] = v;
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

template <typename Row, int TPR, int VPT, bool WIDE>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_forward_kernel(NormArgs a) {
  typedef Cols<Row, TPR, VPT, WIDE> C;
  __shared__ float lds[2][TPR / 64];
  const mlora_norm_block& b = a.b;
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  const int tid = threadIdx.x & (TPR - 1);
  const int64_t row = (int64_t)flat_group() * kRows + threadIdx.x / TPR;
  if (row >= b.n_tokens) return;  // all of a row's threads (one wave, or the workgroup)
  float r[VPT];
  C::load(b.residual, row * b.residual_ld, b.dim, tid, r);
  float wx[VPT];
  if (a.x) C::load_weight(b.x_weight, b.w_dtype, b.weight_offset, b.dim, tid, wx);
  if (b.y) {
    float y[VPT], wy[VPT], gate[VPT], n[VPT];
    C::load(b.y, row * b.y_ld, b.dim, tid, y);
    if (b.y_weight) C::load_weight(b.y_weight, b.w_dtype, b.weight_offset, b.dim, tid, wy);
    C::load_gate(b, row, tid, gate);
    norm_y<C, TPR, VPT>(b, y, wy, lds[0], tid, n);
#pragma unroll
    for (int i = 0; i < VPT; ++i) r[i] = b.residual_scale * r[i] + b.y_scale * gate[i] * n[i];
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) r[i] *= b.residual_scale;
  }
  if (a.r) C::store(a.r, row * a.r_ld, b.dim, tid, r);
  if (!a.x) return;
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) s[0] += r[i] * r[i];
  row_sums<TPR, 1>(s, lds[1], tid);
  const float R = inv_rms(s[0], b.dim, b.eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i) r[i] *= R * wx[i];
  C::store(a.x, row * a.x_ld, b.dim, tid, r);
}

template <typename Row, int TPR, int VPT, bool WIDE>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_backward_kernel(NormArgs a) {
  typedef Cols<Row, TPR, VPT, WIDE> C;
  // of alternate rows: a wave may write the next row's sums while another reads
  __shared__ float sums[2][5][TPR / 64];
  const mlora_norm_block& b = a.b;
  constexpr int kRows = TPR < 256 ? 256 / TPR : 1;
  const int tid = threadIdx.x & (TPR - 1);
  const int D = b.dim;
  const int64_t group = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  const int64_t groups = (int64_t)gridDim.x * kRows;
  float wx[VPT], wy[VPT], sum_wx[VPT], sum_wy[VPT], sum_gate[VPT];
  C::load_weight(b.x_weight, b.w_dtype, b.weight_offset, D, tid, wx);
  if (b.y_weight) C::load_weight(b.y_weight, b.w_dtype, b.weight_offset, D, tid, wy);
#pragma unroll
  for (int i = 0; i < VPT; ++i) sum_wx[i] = sum_wy[i] = sum_gate[i] = 0.f;

  int odd = 0;
  for (int64_t row = group; row < b.n_tokens; row += groups, odd ^= 1) {
    float(*lds)[TPR / 64] = sums[odd];
    float r[VPT], y[VPT], d[VPT], g[VPT], gate[VPT], n[VPT];
    C::load(b.residual, row * b.residual_ld, D, tid, r);
    float Ry = 1.f;
    if (b.y) {
      C::load(b.y, row * b.y_ld, D, tid, y);
      C::load_gate(b, row, tid, gate);
    }
    if (a.d_r) {
      C::load(a.d_r, row * a.d_r_ld, D, tid, d);
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) d[i] = 0.f;
    }
    if (a.d_x) C::load(a.d_x, row * a.d_x_ld, D, tid, g);
    if (b.y) {
      Ry = norm_y<C, TPR, VPT>(b, y, wy, lds[0], tid, n);
#pragma unroll
      for (int i = 0; i < VPT; ++i) r[i] = b.residual_scale * r[i] + b.y_scale * gate[i] * n[i];
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) r[i] *= b.residual_scale;
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
      C::store(a.d_residual, row * a.d_residual_ld, D, tid, out);
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
    if (a.d_y) C::store(a.d_y, row * a.d_y_ld, D, tid, d);
    if (a.d_gate && b.gate_form == kToken && tid == 0)
      static_cast<float*>(a.d_gate)[row * a.d_gate_ld] = s[0];
    if (a.d_gate && b.gate_form == kFull) C::store(a.d_gate, row * a.d_gate_ld, D, tid, n);
  }
  if (a.partial[0]) C::store_f32(a.partial[0] + group * D, D, tid, sum_wx);
  if (a.partial[1]) C::store_f32(a.partial[1] + group * D, D, tid, sum_wy);
  if (a.partial[2]) C::store_f32(a.partial[2] + group * D, D, tid, sum_gate);
}

// Column sums of the groups' partial sums: 32 columns a workgroup, eight
// threads a column.
struct SumArgs {
  const float* partial[kSums];
  float* out[kSums];
  int32_t groups, dim;
};

__global__ void __launch_bounds__(256) norm_sum_kernel(SumArgs a) {
  __shared__ float lds[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  const float* p = a.partial[blockIdx.y];
  float s = 0.f;
  if (a.out[blockIdx.y] && col < a.dim)
    for (int g = part; g < a.groups; g += 8) s += p[(int64_t)g * a.dim + col];
  lds[part][threadIdx.x & 31] = s;
  __syncthreads();
  if (part > 0 || col >= a.dim || !a.out[blockIdx.y]) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += lds[i][threadIdx.x & 31];
  a.out[blockIdx.y][col] = s;
}

// Threads per row and values per thread: the fewest that hold the row.
struct Shape {
  int tpr, vpt;
};
Shape shape_of(int dim) {
  if (dim <= 512) return {64, 8};
  if (dim <= 1024) return {64, 16};
  if (dim <= 2048) return {256, 8};
  if (dim <= 4096) return {256, 16};
  if (dim <= 8192) return {512, 16};
  return {1024, 16};
}
int64_t rows_per_group(Shape s) { return s.tpr < 256 ? 256 / s.tpr : 1; }
// Workgroups of the gradient's kernel.
int64_t backward_grid(int64_t n_tokens, int dim) {
  const int64_t per = rows_per_group(shape_of(dim));
  return std::min<int64_t>((n_tokens + per - 1) / per, kMaxGroups / per);
}

template <typename Row, int TPR, int VPT, bool WIDE>
void launch(const NormArgs& a, bool backward, hipStream_t s) {
  constexpr int threads = TPR < 256 ? 256 : TPR;
  if (backward) {
    hipLaunchKernelGGL((norm_backward_kernel<Row, TPR, VPT, WIDE>),
                       dim3((unsigned)backward_grid(a.b.n_tokens, a.b.dim)), dim3(threads), 0, s, a);
  } else {
    const int64_t per = threads / TPR;
    hipLaunchKernelGGL((norm_forward_kernel<Row, TPR, VPT, WIDE>),
                       flat_grid((a.b.n_tokens + per - 1) / per), dim3(threads), 0, s, a);
  }
}

template <typename Row, bool WIDE>
void launch_shape(const NormArgs& a, bool backward, hipStream_t s) {
  const Shape h = shape_of(a.b.dim);
  if (h.tpr == 64 && h.vpt == 8) return launch<Row, 64, 8, WIDE>(a, backward, s);
  if (h.tpr == 64) return launch<Row, 64, 16, WIDE>(a, backward, s);
  if (h.tpr == 256 && h.vpt == 8) return launch<Row, 256, 8, WIDE>(a, backward, s);
  if (h.tpr == 256) return launch<Row, 256, 16, WIDE>(a, backward, s);
  if (h.tpr == 512) return launch<Row, 512, 16, WIDE>(a, backward, s);
  launch<Row, 1024, 16, WIDE>(a, backward, s);
}

// Whether a matrix (null: any) allows 16-byte accesses.
bool wide_rows(const void* p, int64_t ld, int per) { return !p || (ld % per == 0 && aligned(p, 16)); }

int32_t run(const char* who, const NormArgs& a, bool backward, hipStream_t s) {
  const mlora_norm_block& b = a.b;
  const int per = b.dtype == MLORA_BF16 ? 8 : 4;
  const bool wide =
      b.dim % per == 0 && wide_rows(b.residual, b.residual_ld, per) && wide_rows(b.y, b.y_ld, per) &&
      (b.gate_form == kNoGate || b.gate_form == kToken ||
       wide_rows(b.gate, b.gate_form == kFull ? b.gate_ld : 0, per)) &&
      wide_rows(a.r, a.r_ld, per) && wide_rows(a.x, a.x_ld, per) && wide_rows(a.d_r, a.d_r_ld, per) &&
      wide_rows(a.d_x, a.d_x_ld, per) && wide_rows(a.d_residual, a.d_residual_ld, per) &&
      wide_rows(a.d_y, a.d_y_ld, per) &&
      (b.gate_form != kFull || wide_rows(a.d_gate, a.d_gate_ld, per));
  (void)hipGetLastError();
  if (b.dtype == MLORA_BF16) {
    if (wide)
      launch_shape<Bf16Row, true>(a, backward, s);
    else
      launch_shape<Bf16Row, false>(a, backward, s);
  } else {
    if (wide)
      launch_shape<F32Row, true>(a, backward, s);
    else
      launch_shape<F32Row, false>(a, backward, s);
  }
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
  const uint64_t groups = backward_grid(n_tokens, dim) * rows_per_group(shape_of(dim));
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
    sa.groups = (int32_t)(backward_grid(block->n_tokens, dim) * rows_per_group(shape_of(dim)));
    for (int i = 0; i < kSums; ++i)
      if (sums[i])
        sa.partial[i] = a.partial[i] = static_cast<float*>(workspace) + (int64_t)i * sa.groups * dim;
    if (int32_t rc = run(who, a, true, s)) return rc;
  }
  if (any) {
    sa.dim = dim;
    for (int i = 0; i < kSums; ++i) sa.out[i] = sums[i];
    (void)hipGetLastError();
    hipLaunchKernelGGL(norm_sum_kernel, dim3((dim + 31) / 32, kSums), dim3(256), 0, s, sa);
    return launch_status(who);
  }
  clear_error();
  return MLORA_OK;
}
