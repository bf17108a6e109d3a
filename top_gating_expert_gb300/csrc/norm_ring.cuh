// What the layer norm's kernels share (norm.cu, norm_odd.cu).
#pragma once
#include "elem.cuh"
#include "internal.h"

namespace moe {

// makes a generic lambda's statics one per kernel
template <int N>
struct Tag {};

// g = dy gamma, rounded: contracted into the sum and into g - mean(g) as multiply-adds, the two
// uses would see different values, and a difference that is exactly zero (one column) would
// leave a rounding error times rstd.
__device__ __forceinline__ float product(float a, float b) { return __fmul_rn(a, b); }

constexpr int kRingWarps = 16;
constexpr int kMaxPartials = 160;  // partial column sums of a backward: the workspace holds as many

// 16 bytes of this lane, global to shared, and the groups of such copies.
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Sum of v over the L lanes of a row (a power of two: lanes of one warp, or L / 32 whole warps,
// which then meet at a barrier of their slot's own; s_red: one float a warp of the row, free until
// its next barrier but one). A fixed tree, every lane gets it; all lanes of a warp take part.
template <bool SUB>  // SUB: L < 32
__device__ __forceinline__ float row_lanes_sum(float v, int L, int slot, float* s_red) {
  if constexpr (SUB) {
    for (int off = L >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  } else {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    const int G = L >> 5;
    if (G == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) s_red[(threadIdx.x >> 5) & (G - 1)] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(L) : "memory");
    v = s_red[lane & (G - 1)];
    for (int off = G >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  }
}

constexpr int kFwdStages = 3;

// Warps a row (a power of two up to most) so that NV vectors a lane hold it; 0: too long.
inline int row_warps(int cols, int vec, int nv, int most = 16) {
  int G = 1;
  while (G <= most && int64_t(G) * 32 * vec * nv < cols) G *= 2;
  return G <= most ? G : 0;
}

// Lanes a row: 32 G, or a part of a warp for short rows (several rows a warp).
inline int row_lanes(int cols, int vec, int nv, int G) {
  int L = 32 * G;
  if (G == 1 && nv == 1)
    while (L > 1 && (L / 2) * vec >= cols) L /= 2;
  return L;
}

// Rows of which a smaller part of the slots would take one each all the same: more warps a row
// instead of more pieces a lane. Forward only (1024 x 1003 bf16 6.5 -> 4.9 us, 1024 x 1024 3.6 -> 3.3; where
// it would take a second pass, 1024 x 1024 fp32, 3.2 -> 3.7; the backward writes a partial a CTA, and
// 400 x 1003 fp32 went from 8.0 to 9.4).
inline void spread_rows(int64_t rows, int& nv, int& G) {
  while (nv > 1 && G < kRingWarps && rows <= int64_t(kRingWarps / (2 * G)) * num_sms()) {
    nv /= 2;
    G *= 2;
  }
}

// Rows on no 16-byte boundary (norm_odd.cu). norm_odd_fits: a row of `cols` columns is held whole.
template <typename T>
bool norm_odd_fits(int cols);
template <typename T>
int norm_forward_odd(const moe_norm_t& n, const T* x, const T* res, const float* gamma, const float* beta, T* h,
                     T* y, float* mean, float* rstd, cudaStream_t st);
// nv pieces a lane, G warps a row; the CTAs that wrote a partial to part (null: none wanted) go to *slices
template <typename T>
int norm_backward_odd(const moe_norm_t& n, const T* dy, const T* h, const float* gamma, const float* mean,
                      const float* rstd, const T* dh, T* dx, float* part, int nv, int G, int* slices,
                      cudaStream_t st);

}  // namespace moe
