// Declarations shared by the linear layer's translation units: linear.cu (the C ABI, the
// activation's derivative, the workspace), linear_f32.cu (plain-FMA products) and
// linear_bf16.cu (tcgen05 products).
#pragma once
#include <math.h>

#include "elem.cuh"
#include "internal.h"

namespace moe {

// What a product does with its accumulator v = sum_k A(i, k) B(j, k):
//   pre = v + bias[j];  out = act(pre) + residual.
// ld*: elements between rows i. Null pointers leave their part out.
struct LinearEpi {
  const float* bias = nullptr;
  const void* res = nullptr;
  void* out = nullptr;
  void* pre = nullptr;
  int64_t ldo = 0, ldr = 0, ldp = 0;
  int act = MOE_LIN_NONE;
};

// Partial sums of a split product: at most kPartTiles output tiles of 128 x 128 fp32, by the
// rule that picks the splits (tiles x splits <= kPartTiles when splits > 1).
constexpr int kPartTiles = 304;
constexpr size_t kPartBytes = size_t(kPartTiles) * 128 * 128 * 4;

// out(i, j) over i < rows, j < cols from A(i, k) = A[i * a_i + k * a_k] and B likewise, one
// stride of each operand being 1; part: kPartBytes of scratch.
int launch_linear_f32(const float* A, int64_t a_i, int64_t a_k, const float* B, int64_t b_j,
                      int64_t b_k, int rows, int cols, int K, const LinearEpi& e, float* part,
                      cudaStream_t st);

// A bf16 operand of the tensor-core products: element (r, k) at p[r * ld + k], or with mn at
// p[k * ld + r]; p 16-byte aligned, ld a multiple of 8.
struct LinearOperand {
  const void* p;
  int64_t ld;
  bool mn;
};
int launch_linear_bf16(const LinearOperand& A, const LinearOperand& B, int rows, int cols, int K,
                       const LinearEpi& e, unsigned* status, cudaStream_t st);

#ifdef __CUDACC__
template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  if constexpr (ACT == MOE_LIN_RELU) return v < 0.f ? 0.f : v;  // NaN stays NaN
  if constexpr (ACT == MOE_LIN_GELU) return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
  if constexpr (ACT == MOE_LIN_GELU_TANH) {
    // 0.5 v (1 + tanh(u)) = v sigmoid(2u), u = sqrt(2/pi) (v + 0.044715 v^3)
    const float u = 0.79788456080286536f * (v + 0.044715f * v * v * v);
    return v / (1.f + expf(-2.f * u));
  }
  if constexpr (ACT == MOE_LIN_SILU) return v / (1.f + expf(-v));
  return v;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float v) {
  if constexpr (ACT == MOE_LIN_RELU) return v > 0.f ? 1.f : 0.f;
  if constexpr (ACT == MOE_LIN_GELU)
    return 0.5f * (1.f + erff(v * 0.70710678118654752f)) + v * 0.39894228040143268f * expf(-0.5f * v * v);
  if constexpr (ACT == MOE_LIN_GELU_TANH) {
    // with s = sigmoid(2u): s + v 2u' s (1 - s)
    if (fabsf(v) > 16.f) return v > 0.f ? 1.f : 0.f;  // s (1 - s) is 0 and v^3 may overflow
    const float u2 = 1.59576912160573072f * (v + 0.044715f * v * v * v);
    const float s = 1.f / (1.f + expf(-u2)), t = 1.f / (1.f + expf(u2));
    return s + v * (1.59576912160573072f * (1.f + 0.134145f * v * v)) * s * t;
  }
  if constexpr (ACT == MOE_LIN_SILU) {
    const float s = 1.f / (1.f + expf(-v)), t = 1.f / (1.f + expf(v));
    return s * (1.f + v * t);
  }
  return 1.f;
}

__device__ __forceinline__ float act_any(int act, float v) {
  switch (act) {
    case MOE_LIN_RELU: return act_value<MOE_LIN_RELU>(v);
    case MOE_LIN_GELU: return act_value<MOE_LIN_GELU>(v);
    case MOE_LIN_GELU_TANH: return act_value<MOE_LIN_GELU_TANH>(v);
    case MOE_LIN_SILU: return act_value<MOE_LIN_SILU>(v);
  }
  return v;
}

// f(std::integral_constant-like tag) for the runtime activation
template <int A>
struct ActTag { static constexpr int value = A; };
template <typename F>
int with_act(int act, F&& f) {
  switch (act) {
    case MOE_LIN_NONE: return f(ActTag<MOE_LIN_NONE>{});
    case MOE_LIN_RELU: return f(ActTag<MOE_LIN_RELU>{});
    case MOE_LIN_GELU: return f(ActTag<MOE_LIN_GELU>{});
    case MOE_LIN_GELU_TANH: return f(ActTag<MOE_LIN_GELU_TANH>{});
    case MOE_LIN_SILU: return f(ActTag<MOE_LIN_SILU>{});
  }
  return MOE_ERR_INVALID_ARG;
}
#endif

}  // namespace moe
