// Activations of the gated projections: act(x) = x s(z), s(z) = 1 / (1 + exp(-z)),
//   silu       z = x
//   gelu_tanh  z = 2 sqrt(2 / pi) (x + 0.044715 x^3), since
//              (1 + tanh(z / 2)) / 2 = s(z)
// and their slopes s + x s (1 - s) z'.  Two special-function operations each, in
// FP32, far below the BF16 rounding of what follows (tanh.approx would take one,
// but is off by 2^-11).  z's roundings move s by (1 - s) 2^-21 |z|, relative to s, at most
// (silu: a quarter of that), the two operations and the sum by 2^-21 more: a gate of -1
// has s to 2^-19, the last ones whose s is a normal number (z = -87) to 2^-14.  -inf as a
// gate gives NaN (0 times inf), as the formula does; so does the slope of +inf.
#pragma once

#include "gb300gemm.h"
#include "ptx.cuh"

namespace gb300 {

template <int kAct>
struct ActKind {
  static constexpr int value = kAct;
};

// -z log2 e of act kind kAct
template <int kAct>
__device__ __forceinline__ float gate_exponent(float x) {
  constexpr float kL = -1.4426950408889634f;
  if constexpr (kAct == GEMM_ACT_SILU) return kL * x;
  constexpr float kC = 1.5957691216057308f * kL;  // 2 sqrt(2 / pi)
  return x * (kC + kC * 0.044715f * (x * x));
}

template <int kAct>
__device__ __forceinline__ float gate_act(float x) {
  return x * ptx::rcp(1.0f + ptx::ex2(gate_exponent<kAct>(x)));
}

// (act(x), its slope)
template <int kAct>
__device__ __forceinline__ float2 gate_act_slope(float x) {
  const float s = ptx::rcp(1.0f + ptx::ex2(gate_exponent<kAct>(x)));
  float dz = 1.0f;
  // (past |x| = 100, where s (1 - s) is zero, z' stays finite)
  if constexpr (kAct == GEMM_ACT_GELU_TANH)
    dz = 1.5957691216057308f * (1.0f + 3.0f * 0.044715f * fminf(x * x, 1e4f));
  return make_float2(x * s, s + x * s * (1.0f - s) * dz);
}

}  // namespace gb300
