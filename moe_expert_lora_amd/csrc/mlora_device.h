// Device and launch helpers shared by the MoE-layer operators around the fold
// (mlora_moe.hip, mlora_w4.hip).
#ifndef MLORA_DEVICE_H_
#define MLORA_DEVICE_H_

#include <hip/hip_runtime.h>

#include <cstdint>

#include "mlora.h"
#include "mlora_internal.h"

namespace mlora {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Two fp32 -> two bf16 in one word (low half = a), round to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
// bf16 pair word -> its low / high value as fp32 (exact).
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A value every lane of the wave holds, moved to a scalar register.
__device__ __forceinline__ int uniform_i32(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Element types of a row: how many fit 16 bytes, and the exact widening /
// one round-to-nearest-even narrowing of a 16-byte chunk or one element.
struct Bf16Row {
  typedef uint16_t elem;
  static constexpr int kPer16 = 8;
  static __device__ __forceinline__ float widen(elem v) {
    return __uint_as_float((uint32_t)v << 16);
  }
  static __device__ __forceinline__ elem narrow(float f) { return (elem)pack_bf16(f, 0.f); }
  static __device__ __forceinline__ void widen16(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = lo_f(v[i]);
      f[2 * i + 1] = hi_f(v[i]);
    }
  }
  static __device__ __forceinline__ u32x4 narrow16(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    return v;
  }
};
struct F32Row {
  typedef float elem;
  static constexpr int kPer16 = 4;
  static __device__ __forceinline__ float widen(elem v) { return v; }
  static __device__ __forceinline__ elem narrow(float f) { return f; }
  static __device__ __forceinline__ void widen16(u32x4 v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
  static __device__ __forceinline__ u32x4 narrow16(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
    return v;
  }
};

// x rotated by N lanes within each row of 16 lanes (one DPP move).
template <int N>
__device__ __forceinline__ uint32_t ror16(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + N, 0xf, 0xf, false);
}
// The value of the lane 16 (32) away in the other row (half) of the wave's row
// pair (halves), beside the lane's own, in an order both lanes agree on.
__device__ __forceinline__ u32x2 pair_rows(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return u32x2{(uint32_t)r[0], (uint32_t)r[1]};
}
__device__ __forceinline__ u32x2 pair_halves(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return u32x2{(uint32_t)r[0], (uint32_t)r[1]};
}

// Reductions over the LPT lanes (16, 32 or 64) that share a row; every lane
// gets the result. Four rotations inside rows of 16, then the rows in pairs,
// then the halves. The order is fixed.
template <int LPT, typename T, typename Op>
__device__ __forceinline__ T group_reduce(T v, Op op) {
  auto bits = [](T x) { return __builtin_bit_cast(uint32_t, x); };
  auto from = [](uint32_t x) { return __builtin_bit_cast(T, x); };
  v = op(v, from(ror16<8>(bits(v))));
  v = op(v, from(ror16<4>(bits(v))));
  v = op(v, from(ror16<2>(bits(v))));
  v = op(v, from(ror16<1>(bits(v))));
  if constexpr (LPT >= 32) {
    const u32x2 r = pair_rows(bits(v));
    v = op(from(r[0]), from(r[1]));
  }
  if constexpr (LPT == 64) {
    const u32x2 r = pair_halves(bits(v));
    v = op(from(r[0]), from(r[1]));
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int LPT>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return group_reduce<LPT>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<LPT>(v, [](float a, float b) { return a + b; });
}

// LDS traffic of one wave is in order; this keeps the compiler from moving
// accesses across, where lanes of a wave read what other lanes wrote.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// A grid of any number of workgroups. HIP takes fewer than 2^32 threads along one
// dimension: from kGridRow workgroups (of up to 256 threads) on, further rows lie
// along y, the last of them with workgroups past the end.
constexpr int kGridRow = 1 << 23;
inline dim3 flat_grid(int64_t workgroups) {
  if (workgroups <= kGridRow) return dim3((unsigned)workgroups);
  return dim3(kGridRow, (unsigned)((workgroups + kGridRow - 1) / kGridRow));
}
// The workgroup's number in it.
__device__ __forceinline__ int flat_group() { return (int)(blockIdx.y * kGridRow + blockIdx.x); }

inline int32_t launch_status(const char* who) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MLORA_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
  clear_error();
  return MLORA_OK;
}

inline bool aligned(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// Largest token, slot or row count of one call.
constexpr int64_t kMaxRows = 0x3fffffffll;

}  // namespace mlora

#endif  // MLORA_DEVICE_H_
