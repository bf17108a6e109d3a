// Loads and stores of the two element types (float, bf16) as fp32, shared by the norm and
// linear kernels.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace moe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// the hardware's exp2 and reciprocal (2 and 1 ulp; denormals are zero)
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// the largest of three in one instruction (a NaN is left out, as in fmaxf)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Pairs of fp32 in one 64-bit register: two operations an instruction, each rounded as alone.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 set2(float v) { return pack2(v, v); }

// VEC elements as one access: 16 bytes, or a single element.
template <typename T, int VEC>
struct Vec {
  T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load_vec(const T* p) {
  Vec<T, VEC> r;
  if constexpr (VEC * sizeof(T) == 16) *reinterpret_cast<uint4*>(r.v) = *reinterpret_cast<const uint4*>(p);
  else r.v[0] = *p;
  return r;
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, VEC>& r) {
  if constexpr (VEC * sizeof(T) == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(r.v);
  else *p = r.v[0];
}
// the same from shared memory, where a piece is 16 or 4 bytes
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> load_piece(const void* p) {
  return load_vec<T, VEC>(static_cast<const T*>(p));
}
// VEC floats from a 16-byte aligned address (VEC 4 or 8), or one
template <int VEC>
__device__ __forceinline__ void load_floats(const float* p, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = __ldg(p);
  } else {
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) reinterpret_cast<float4*>(f)[q] = __ldg(reinterpret_cast<const float4*>(p) + q);
  }
}

// Sum over the block of NW warps of one float per thread, valid in every thread; the order
// is a fixed tree. s_red: NW floats that no thread uses until the next barrier.
template <int NW>
__device__ __forceinline__ float block_sum_all(float v, float* s_red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if constexpr (NW == 1) return v;
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) r += s_red[w];
  return r;
}


// Column sums of partial results: value(s, c) over s < n, for 32 columns from c0 on, by a CTA of 32
// warps: each warp every 32nd s (a lane a column), then warp w joins column w's 32 sums. The order
// depends on n alone. (Eight warps took twice the time: the loads of one warp are one chain.)
template <typename Value, typename Store>
__device__ __forceinline__ void column_sums(int n, int c0, int cols, float (*s_part)[33], Value&& value,
                                            Store&& store) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float t = 0.f;
  if (c0 + lane < cols) {
#pragma unroll 8
    for (int s = warp; s < n; s += 32) t += value(s, c0 + lane);
  }
  s_part[warp][lane] = t;
  __syncthreads();
  t = s_part[lane][warp];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  if (lane == 0 && c0 + warp < cols) store(c0 + warp, t);
}

}  // namespace moe
