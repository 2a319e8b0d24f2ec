// The router's choice of a token's experts, held in the lanes of a wave: shared
// by the router's kernels (mlora_moe.hip) and the layer's (mlora_layer.hip).
#ifndef MLORA_ROUTER_H_
#define MLORA_ROUTER_H_

#include "mlora_device.h"

namespace mlora {

// w_j = softmax(l)[i_j] over the k largest logits l[i_0] >= l[i_1] >= ..., ties
// to the lowest index. LPT lanes hold one token's row in registers (VPL values
// a lane); k times, the row's largest key is found by a reduction over those
// lanes and taken out. A key orders like the value: the float's bits with the
// sign folded in, -0 taken as +0, a NaN above every number, 0 for no value.
// A bf16 key has 16 bits, so the inverted index fits below it: one word finds
// value and index in one reduction; an fp32 key takes a second one for the
// index. The chosen logits stay in lanes 0..k-1.

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;
constexpr float kNegInf = -__builtin_inff();

// Float bits -> order-preserving key (bits 0x007FFFFF for -inf, never 0).
__device__ __forceinline__ uint32_t order_key(uint32_t u) {
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if (u == 0x80000000u) u = 0;
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// Expert of value j of lane gl: VEC neighbours, lanes in turn. WIDE rows move
// those neighbours in one access, others one by one; the sums' order, and so
// the bits of the result, are the same.
template <int LPT, int VEC>
__device__ __forceinline__ int expert_of(int j, int gl) {
  return (j / VEC) * (LPT * VEC) + gl * VEC + j % VEC;
}

// One token's row: value j of a lane is expert_of(j), 0 past E.
template <typename Row, int LPT, int VPL, int VEC, bool WIDE>
__device__ __forceinline__ void load_row(const void* base, int64_t off, int E, int gl,
                                         float (&v)[VPL]) {
  const typename Row::elem* p = static_cast<const typename Row::elem*>(base) + off;
#pragma unroll
  for (int j = 0; j < VPL; j += VEC) {
    const int e = expert_of<LPT, VEC>(j, gl);
    if constexpr (!WIDE) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j + i] = e + i < E ? Row::widen(p[e + i]) : 0.f;
    } else {
      typedef typename Row::elem vec __attribute__((ext_vector_type(VEC)));
      vec w = {};
      if (e < E) w = *reinterpret_cast<const vec*>(p + e);
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[j + i] = Row::widen(w[i]);
    }
  }
}

// The k largest values of the row that load_row put into v: lane gl < k returns
// the j = gl-th one's softmax weight and its expert in *mine_e.
template <typename Row, int LPT, int VPL, int VEC>
__device__ __forceinline__ float choose_experts(const float (&v)[VPL], int E, int k, bool renorm,
                                                int gl, int* mine_e) {
  constexpr bool kPacked = sizeof(typename Row::elem) == 2;
  uint32_t key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = expert_of<LPT, VEC>(j, gl);
    const uint32_t u = order_key(__float_as_uint(v[j]));
    key[j] = e < E ? (kPacked ? (u & 0xffff0000u) | (0xffffu - e) : u) : 0u;
  }

  float top = 0.f, sum = 0.f, mine = 0.f;
  *mine_e = 0;
  for (int it = 0; it < k; ++it) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) m = max(m, key[j]);
    m = group_max<LPT>(m);
    int e;
    if constexpr (kPacked) {
      e = 0xffff - (int)(m & 0xffffu);
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = key[j] == m ? 0u : key[j];
    } else {
      uint32_t c = 0xffffffffu;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        c = min(c, key[j] == m ? (uint32_t)expert_of<LPT, VEC>(j, gl) : 0xffffffffu);
      e = (int)group_min<LPT>(c);
#pragma unroll
      for (int j = 0; j < VPL; ++j) key[j] = expert_of<LPT, VEC>(j, gl) == e ? 0u : key[j];
    }
    const float val = key_value(kPacked ? ((m >> 16) == 0xffffu ? 0xffffffffu : (m & 0xffff0000u) |
                                                        ((m >> 31) ? 0u : 0xffffu))
                                        : m);
    if (it == 0) {
      top = val;
      if (!renorm) {
        // the softmax's sum over every expert, about the row's maximum
#pragma unroll
        for (int j = 0; j < VPL; ++j)
          sum += expert_of<LPT, VEC>(j, gl) < E ? expf(v[j] - top) : 0.f;
        sum = group_sum<LPT>(sum);
      }
    }
    if (gl == it) {
      mine = val;
      *mine_e = e;
    }
  }
  float w = gl < k ? expf(mine - top) : 0.f;
  if (renorm) sum = group_sum<LPT>(w);
  // a row with every expert masked (-inf): no probabilities; weights of 0
  return top == kNegInf ? 0.f : w / sum;
}

}  // namespace mlora

#endif  // MLORA_ROUTER_H_
