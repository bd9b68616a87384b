// Activations of the gated feed-forward block and their slopes, shared by its kernels.
//   SILU a(g) = g p, p = 1 / (1 + e^-g);           a' = p + a (1 - p)
//   GELU a(g) = g p, p = 1 / (1 + e^-u),           a' = p + a (1 - p) u'
//        u = 2 sqrt(2/pi) (g + 0.044715 g^3): 0.5 g (1 + tanh(u / 2)) written with one exponential
//   RELU a(g) = g and a' = 1 where g > 0, else 0 (of NaN too, as the library's ReLU has it)
#pragma once

#include "kernels.hpp"

namespace gek {

enum Gate { GATE_SILU = 0, GATE_GELU = 1, GATE_RELU = 2 };

// 1 / (1 + 2^t). FINE (fp32 results): the library's exp2 and an exact division; otherwise the
// hardware's exp2 and reciprocal, within a few units of fp32 and far below 16-bit rounding.
template <bool FINE>
__device__ __forceinline__ float inv_1p_exp2(float t) {
  if constexpr (FINE) return 1.0f / (1.0f + exp2f(t));
  else return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}
// 1 / (1 + e^-g). (FINE takes e^x of the argument itself: rounding log2(e) g first would cost
// |g| units in the last place.)
template <bool FINE>
__device__ __forceinline__ float logistic(float g) {
  if constexpr (FINE) return 1.0f / (1.0f + expf(-g));
  else return inv_1p_exp2<false>(-1.4426950408889634f * g);
}

constexpr float kGelu1 = 1.5957691216057308f;     // 2 sqrt(2/pi)
constexpr float kGelu3 = 0.07135481282553734f;    // 0.044715 of it

template <int ACT, bool FINE>
__device__ __forceinline__ float gate_act(float g) {
  if constexpr (ACT == GATE_RELU) return g > 0.0f ? g : 0.0f;
  else if constexpr (ACT == GATE_SILU) return g * logistic<FINE>(g);
  else return g * logistic<FINE>(g * __builtin_fmaf(kGelu3, g * g, kGelu1));
}

// a and a' together.
template <int ACT, bool FINE>
__device__ __forceinline__ void gate_slope(float g, float& a, float& da) {
  if constexpr (ACT == GATE_RELU) {
    a = g > 0.0f ? g : 0.0f;
    da = g > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == GATE_SILU) {
    const float p = logistic<FINE>(g);
    a = g * p;
    da = __builtin_fmaf(a, 1.0f - p, p);
  } else {
    const float g2 = fminf(g * g, 1e8f);   // p (1 - p) is 0 long before: keeps 0 times u' from 0 times infinity
    const float p = logistic<FINE>(g * __builtin_fmaf(kGelu3, g * g, kGelu1));
    a = g * p;
    da = __builtin_fmaf(a * (1.0f - p), __builtin_fmaf(3.0f * kGelu3, g2, kGelu1), p);
  }
}

// f with the activation as a compile-time constant.
template <class F>
__device__ __forceinline__ void with_gate(int act, F&& f) {
  if (act == GATE_SILU) f(std::integral_constant<int, GATE_SILU>{});
  else if (act == GATE_GELU) f(std::integral_constant<int, GATE_GELU>{});
  else f(std::integral_constant<int, GATE_RELU>{});
}

}  // namespace gek
