// tq_ffn.h -- device helpers shared by the gated feed-forward and adapter
// kernels: bf16 conversions, the gate activations and their derivatives.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint32_t bits) { return __uint_as_float(bits << 16); }

// Round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

constexpr int kActSilu = 0, kActGelu = 1;

// sigma(z) = 1 / (1 + e^-z); e^-z overflows to infinity and the quotient to 0.
// v_rcp_f32 is within one unit of fp32; a correctly rounded division costs
// ten instructions more, a fifth of the forward kernel's epilogue.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// GELU in its tanh form: g (1 + tanh z) / 2 = g sigma(2z), z = c (g + a g^3).
constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
  if constexpr (ACT == kActSilu) return g * sigmoid(g);
  return g * sigmoid(2.0f * kGeluC * (g + kGeluA * g * g * g));
}

// act(g) and act'(g).  silu' = s (1 + g (1 - s)).  gelu' = s + 2 g s (1 - s)
// z'(g); where s (1 - s) has vanished the second term is 0 (z' may have
// overflowed there).
template <int ACT>
__device__ __forceinline__ void act_and_slope(float g, float &value, float &slope) {
  if constexpr (ACT == kActSilu) {
    const float s = sigmoid(g);
    value = g * s;
    slope = s * (1.0f + g * (1.0f - s));
  } else {
    const float s = sigmoid(2.0f * kGeluC * (g + kGeluA * g * g * g));
    const float v = s * (1.0f - s);
    value = g * s;
    slope = s + (v == 0.0f ? 0.0f : 2.0f * g * v * (kGeluC * (1.0f + 3.0f * kGeluA * g * g)));
  }
}

}  // namespace tq
