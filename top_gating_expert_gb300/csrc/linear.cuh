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
// rule that picks the splits (tiles x splits <= kPartTiles when splits > 1; more of smaller tiles).
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

// The forward for one bf16 or up to eight fp32 tokens, operands on any boundary.
int launch_linear_few(int bf16, const void* x, int64_t ldx, const void* W, int64_t ldw, int T, int N, int K,
                      const LinearEpi& e, cudaStream_t st);

#ifdef __CUDACC__
template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  if constexpr (ACT == MOE_LIN_RELU) return v < 0.f ? 0.f : v;  // NaN stays NaN
  if constexpr (ACT == MOE_LIN_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);  // the tail exact
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
    return 0.5f * erfcf(v * -0.70710678118654752f) + v * 0.39894228040143268f * expf(-0.5f * v * v);
  if constexpr (ACT == MOE_LIN_GELU_TANH) {
    // with s = sigmoid(2u): s + v 2u' s (1 - s)
    if (fabsf(v) > 16.f) return v > 0.f ? 1.f : 0.f;  // s (1 - s) is 0 and v^3 may overflow
    const float u2 = 1.5957691216f * (v + 0.044715f * v * v * v);
    const float s = 1.f / (1.f + expf(-u2)), t = 1.f / (1.f + expf(u2));
    return s + v * (1.5957691216f * (1.f + 0.134145f * v * v)) * s * t;
  }
  if constexpr (ACT == MOE_LIN_SILU) {
    const float s = 1.f / (1.f + expf(-v)), t = 1.f / (1.f + expf(v));
    return s * (1.f + v * t);
  }
  return 1.f;
}

// The same for results that are rounded to bf16 (2^-8): hardware exponential and reciprocal (a
// few ulp), and for the normal distribution function
//   Phi(-|v|) = erfc(x) / 2, x = |v| / sqrt(2), erfc(x) = exp(-x^2) R(t), t = 1 / (1 + 0.38 x),
// with R a polynomial of degree 7 without constant term fitted to exp(x^2) erfc(x) by linear
// programming on the relative error over 0 <= x <= 10 (1.0e-6; the tail keeps its relative
// precision). erff's two branches and 1 + erf's cancellation cost about twice the instructions, and
// pairs in one instruction halve what is left (the 8192 x 14336 epilogue and the backward's pass
// over dy and pre are bound by issue).
// All on pairs. e = exp(-v^2 / 2), and Phi(v): the tail below zero, one less it above
__device__ __forceinline__ f32x2 exp2_2(f32x2 x) {
  const float2 f = unpack2(x);
  return pack2(exp2_approx(f.x), exp2_approx(f.y));
}
__device__ __forceinline__ f32x2 rcp_2(f32x2 x) {
  const float2 f = unpack2(x);
  return pack2(rcp_approx(f.x), rcp_approx(f.y));
}
__device__ __forceinline__ f32x2 normal_cdf2(f32x2 v, f32x2& e) {
  const float2 f = unpack2(v);
  e = exp2_2(mul2(mul2(v, v), set2(-0.72134752044448170f)));
  const f32x2 t = rcp_2(fma2(pack2(fabsf(f.x), fabsf(f.y)), set2(0.26870057685f), set2(1.f)));
  f32x2 r = set2(-0.0625806375f);  // R's coefficients, halved
  r = fma2(r, t, set2(0.167536944f));
  r = fma2(r, t, set2(-0.03422876445f));
  r = fma2(r, t, set2(0.123351455f));
  r = fma2(r, t, set2(0.0905347165f));
  r = fma2(r, t, set2(0.108237808f));
  r = fma2(r, t, set2(0.1071479915f));
  const f32x2 tail = mul2(e, mul2(r, t));
  const float2 lo = unpack2(tail), hi = unpack2(fma2(tail, set2(-1.f), set2(1.f)));
  return pack2(f.x < 0.f ? lo.x : hi.x, f.y < 0.f ? lo.y : hi.y);
}
template <int ACT>
__device__ __forceinline__ f32x2 act_fast2(f32x2 v) {
  constexpr float kL2e = 1.44269504088896341f;
  if constexpr (ACT == MOE_LIN_GELU) {
    f32x2 e;
    return mul2(v, normal_cdf2(v, e));
  } else if constexpr (ACT == MOE_LIN_GELU_TANH) {  // v / (1 + exp(-2u))
    const f32x2 u = mul2(v, fma2(mul2(v, v), set2(-0.0713548162726f * kL2e), set2(-1.59576912160573f * kL2e)));
    return mul2(v, rcp_2(add2(exp2_2(u), set2(1.f))));
  } else if constexpr (ACT == MOE_LIN_SILU) {
    return mul2(v, rcp_2(add2(exp2_2(mul2(v, set2(-kL2e))), set2(1.f))));
  } else {
    const float2 f = unpack2(v);
    return pack2(act_value<ACT>(f.x), act_value<ACT>(f.y));
  }
}
template <int ACT>
__device__ __forceinline__ f32x2 slope_fast2(f32x2 v) {
  constexpr float kL2e = 1.44269504088896341f;
  const float2 f = unpack2(v);
  if constexpr (ACT == MOE_LIN_GELU) {
    f32x2 e;
    const f32x2 phi = normal_cdf2(v, e);
    return fma2(mul2(v, set2(0.39894228040143268f)), e, phi);
  } else if constexpr (ACT == MOE_LIN_GELU_TANH) {
    const f32x2 v2 = mul2(v, v);  // the exponent capped at 2^115: the reciprocal stays normal
    const float2 u = unpack2(mul2(v, fma2(v2, set2(-0.0713548162726f * kL2e), set2(-1.59576912160573f * kL2e))));
    const f32x2 e = pack2(exp2_approx(fminf(u.x, 115.f)), exp2_approx(fminf(u.y, 115.f)));
    const f32x2 s = rcp_2(add2(e, set2(1.f)));
    const float2 d = unpack2(
        fma2(mul2(v, fma2(v2, set2(0.214064448818f), set2(1.59576912160573f))), mul2(s, mul2(e, s)), s));
    // far out v^3 may overflow; the slope is 0 or 1 there
    return pack2(fabsf(f.x) > 16.f ? (f.x > 0.f ? 1.f : 0.f) : d.x, fabsf(f.y) > 16.f ? (f.y > 0.f ? 1.f : 0.f) : d.y);
  } else if constexpr (ACT == MOE_LIN_SILU) {
    const float2 u = unpack2(mul2(v, set2(-kL2e)));
    const f32x2 e = pack2(exp2_approx(fminf(u.x, 115.f)), exp2_approx(fminf(u.y, 115.f)));
    const f32x2 s = rcp_2(add2(e, set2(1.f)));
    return mul2(s, fma2(v, mul2(e, s), set2(1.f)));
  } else {
    return pack2(act_slope<ACT>(f.x), act_slope<ACT>(f.y));
  }
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
// N values at once, the activation chosen outside the loop
template <int ACT, int N>
__device__ __forceinline__ void act_pairs(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 f = unpack2(act_fast2<ACT>(pack2(v[i], v[i + 1])));
    v[i] = f.x;
    v[i + 1] = f.y;
  }
}
template <int N>
__device__ __forceinline__ void act_fast_all(int act, float (&v)[N]) {
  switch (act) {
    case MOE_LIN_RELU: act_pairs<MOE_LIN_RELU>(v); break;
    case MOE_LIN_GELU: act_pairs<MOE_LIN_GELU>(v); break;
    case MOE_LIN_GELU_TANH: act_pairs<MOE_LIN_GELU_TANH>(v); break;
    case MOE_LIN_SILU: act_pairs<MOE_LIN_SILU>(v); break;
  }
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
