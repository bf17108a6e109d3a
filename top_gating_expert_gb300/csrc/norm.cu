// Layer norm over the columns of a row-major matrix, forward and backward.
//
//   forward   h = x (+ residual); y = (h - mean) rstd gamma (+ beta), rstd = 1/sqrt(var + eps)
//   backward  xh = (h - mean) rstd, g = dy gamma:
//             dx = rstd (g - mean(g) - xh mean(g xh)) (+ dh)
//             dgamma = sum_rows dy xh, dbeta = sum_rows dy
//
// The variance is the mean of the squared deviations from the mean already formed (not
// E[h^2] - mean^2, which cancels when a channel's offset is large against its spread). Both
// directions are bound by memory: every input is read once and every output written once.
#include <algorithm>

#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreadsN = 256;
constexpr int kWarpsN = kThreadsN / 32;

// One CTA a row, any length and alignment: three walks over the row (sum, squared
// deviations, output), the later two from cache.
template <typename T>
__global__ void __launch_bounds__(kThreadsN)
    norm_fwd_any_kernel(const T* x, const T* res, const float* __restrict__ gamma,
                        const float* __restrict__ beta, T* h, T* y, float* mean, float* rstd,
                        moe_norm_t n) {
  __shared__ float s_red[2 * kWarpsN];
  pdl_wait();
  pdl_trigger();
  const int64_t r = blockIdx.x;
  const int M = n.cols;
  const T* xr = x + r * n.ldx;
  const T* rr = res ? res + r * n.ldr : nullptr;
  float s = 0.f;
  for (int i = threadIdx.x; i < M; i += kThreadsN) s += to_f32(xr[i]) + (rr ? to_f32(rr[i]) : 0.f);
  const float mu = block_sum_all<kWarpsN>(s, s_red) / float(M);
  float v = 0.f;
  for (int i = threadIdx.x; i < M; i += kThreadsN) {
    const float d = to_f32(xr[i]) + (rr ? to_f32(rr[i]) : 0.f) - mu;
    v = fmaf(d, d, v);
  }
  const float rs = 1.f / sqrtf(block_sum_all<kWarpsN>(v, s_red + kWarpsN) / float(M) + n.eps);
  for (int i = threadIdx.x; i < M; i += kThreadsN) {
    const float hv = to_f32(xr[i]) + (rr ? to_f32(rr[i]) : 0.f);
    const float o = fmaf((hv - mu) * rs, gamma[i], beta ? beta[i] : 0.f);
    if (h) h[r * n.ldh + i] = from_f32<T>(hv);
    y[r * n.ldy + i] = from_f32<T>(o);
  }
  if (threadIdx.x == 0) {
    if (mean) mean[r] = mu;
    if (rstd) rstd[r] = rs;
  }
}

// g = dy gamma, rounded: contracted into the sum and into g - mean(g) as multiply-adds, the two
// uses would see different values, and a difference that is exactly zero (one column) would
// leave a rounding error times rstd.
__device__ __forceinline__ float product(float a, float b) { return __fmul_rn(a, b); }

// One CTA a row: the two row sums, then dx.
template <typename T>
__global__ void __launch_bounds__(kThreadsN)
    norm_bwd_dx_any_kernel(const T* dy, const T* __restrict__ h, const float* __restrict__ gamma,
                           const float* __restrict__ mean, const float* __restrict__ rstd,
                           const T* dh, T* dx, moe_norm_t n) {
  __shared__ float s_red[2 * kWarpsN];
  pdl_wait();
  pdl_trigger();
  const int64_t r = blockIdx.x;
  const int M = n.cols;
  const T* hr = h + r * n.ldx;
  const T* dr = dy + r * n.ldy;
  const float mu = mean[r], rs = rstd[r];
  float s1 = 0.f, s2 = 0.f;
  for (int i = threadIdx.x; i < M; i += kThreadsN) {
    const float g = product(to_f32(dr[i]), gamma[i]);
    s1 += g;
    s2 = fmaf(g, (to_f32(hr[i]) - mu) * rs, s2);
  }
  s1 = block_sum_all<kWarpsN>(s1, s_red) / float(M);
  s2 = block_sum_all<kWarpsN>(s2, s_red + kWarpsN) / float(M);
  for (int i = threadIdx.x; i < M; i += kThreadsN) {
    const float g = product(to_f32(dr[i]), gamma[i]);
    const float xh = (to_f32(hr[i]) - mu) * rs;
    float o = rs * (g - s1 - xh * s2);
    if (dh) o += to_f32(dh[r * n.ldr + i]);
    dx[r * n.ldh + i] = from_f32<T>(o);
  }
}

// Partial column sums of dy * xh and dy: CTA (c, s) takes 32 columns and row slice s; its
// eight warps walk the slice's rows, then add in order.
constexpr int kSliceCols = 32;

template <typename T>
__global__ void __launch_bounds__(kThreadsN)
    norm_bwd_cols_any_kernel(const T* __restrict__ dy, const T* __restrict__ h,
                             const float* __restrict__ mean, const float* __restrict__ rstd,
                             float* part, int slice, moe_norm_t n) {
  __shared__ float s_g[kWarpsN][32], s_b[kWarpsN][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * kSliceCols + lane;
  const int64_t r0 = int64_t(blockIdx.y) * slice, r1 = min(int64_t(n.rows), r0 + slice);
  float g = 0.f, b = 0.f;
  if (c < n.cols)
    for (int64_t r = r0 + warp; r < r1; r += kWarpsN) {
      const float d = to_f32(dy[r * n.ldy + c]);
      g = fmaf(d, (to_f32(h[r * n.ldx + c]) - mean[r]) * rstd[r], g);
      b += d;
    }
  s_g[warp][lane] = g;
  s_b[warp][lane] = b;
  __syncthreads();
  if (warp == 0 && c < n.cols) {
    for (int w = 1; w < kWarpsN; ++w) {
      g += s_g[w][lane];
      b += s_b[w][lane];
    }
    part[(int64_t(blockIdx.y) * 2) * n.cols + c] = g;
    part[(int64_t(blockIdx.y) * 2 + 1) * n.cols + c] = b;
  }
}

// dgamma and dbeta from the slices' partials [slices][2][cols], added in slice order.
__global__ void __launch_bounds__(kThreadsN)
    norm_bwd_sum_kernel(const float* __restrict__ part, int slices, int cols, float* dgamma,
                        float* dbeta) {
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x * kThreadsN + threadIdx.x;
  if (c >= cols) return;
  float g = 0.f, b = 0.f;
  for (int s = 0; s < slices; ++s) {
    g += part[int64_t(s) * 2 * cols + c];
    b += part[(int64_t(s) * 2 + 1) * cols + c];
  }
  if (dgamma) dgamma[c] = g;
  if (dbeta) dbeta[c] = b;
}

constexpr int kMaxSlices = 304;

int check_norm(const moe_norm_t* n) {
  if (!n || n->rows < 0 || n->cols < 1 || !(n->eps >= 0.f) || n->eps > 3.0e38f) return MOE_ERR_INVALID_ARG;
  if (n->dtype != MOE_F32 && n->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  const int64_t M = n->cols;
  if (n->ldx < M || n->ldr < M || n->ldh < M || n->ldy < M) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

size_t norm_ws_bytes(const moe_norm_t& n) {
  return 256 + align256(size_t(kMaxSlices) * 2 * size_t(n.cols) * 4);
}

template <typename T>
int norm_forward_t(const moe_norm_t& n, const void* x, const void* residual, const float* gamma,
                   const float* beta, void* h, void* y, float* mean, float* rstd, cudaStream_t st) {
  return launch_kernel(norm_fwd_any_kernel<T>, dim3(unsigned(n.rows)), dim3(kThreadsN), 0, st,
                       static_cast<const T*>(x), static_cast<const T*>(residual), gamma, beta,
                       static_cast<T*>(h), static_cast<T*>(y), mean, rstd, n);
}

template <typename T>
int norm_backward_t(const moe_norm_t& n, const void* dy, const void* h, const float* gamma,
                    const float* mean, const float* rstd, const void* dh, void* dx, float* dgamma,
                    float* dbeta, char* ws, cudaStream_t st) {
  const T* dyt = static_cast<const T*>(dy);
  const T* ht = static_cast<const T*>(h);
  int rc;
  if (dgamma || dbeta) {  // before dx, which may be written over dy
    const int cblocks = (n.cols + kSliceCols - 1) / kSliceCols;
    int slices = std::min(kMaxSlices, std::max(1, 8 * num_sms() / cblocks));
    slices = std::min(slices, (n.rows + kWarpsN - 1) / kWarpsN);
    const int slice = (n.rows + slices - 1) / slices;
    slices = (n.rows + slice - 1) / slice;
    float* part = reinterpret_cast<float*>(ws + 256);
    if ((rc = launch_kernel(norm_bwd_cols_any_kernel<T>, dim3(unsigned(cblocks), unsigned(slices)),
                            dim3(kThreadsN), 0, st, dyt, ht, mean, rstd, part, slice, n)) != MOE_OK)
      return rc;
    if ((rc = launch_kernel(norm_bwd_sum_kernel, dim3(unsigned((n.cols + kThreadsN - 1) / kThreadsN)),
                            dim3(kThreadsN), 0, st, static_cast<const float*>(part), slices, n.cols,
                            dgamma, dbeta)) != MOE_OK)
      return rc;
  }
  return launch_kernel(norm_bwd_dx_any_kernel<T>, dim3(unsigned(n.rows)), dim3(kThreadsN), 0, st, dyt,
                       ht, gamma, mean, rstd, static_cast<const T*>(dh), static_cast<T*>(dx), n);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_norm_forward(const moe_norm_t* n, const void* x, const void* residual, const float* gamma,
                     const float* beta, void* h, void* y, float* mean, float* rstd,
                     moe_stream_t stream) {
  const int rc = check_norm(n);
  if (rc != MOE_OK) return rc;
  if (n->rows == 0) return MOE_OK;
  if (!x || !gamma || !y) return MOE_ERR_INVALID_ARG;
  if (h && h == y) return MOE_ERR_INVALID_ARG;
  return n->dtype == MOE_F32
             ? norm_forward_t<float>(*n, x, residual, gamma, beta, h, y, mean, rstd, stream)
             : norm_forward_t<__nv_bfloat16>(*n, x, residual, gamma, beta, h, y, mean, rstd, stream);
}

int moe_norm_workspace_bytes(const moe_norm_t* n, size_t* bytes) {
  const int rc = check_norm(n);
  if (rc != MOE_OK) return rc;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = norm_ws_bytes(*n);
  return MOE_OK;
}

int moe_norm_backward(const moe_norm_t* n, const void* dy, const void* h, const float* gamma,
                      const float* mean, const float* rstd, const void* dh, void* dx,
                      float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                      moe_stream_t stream) {
  const int rc = check_norm(n);
  if (rc != MOE_OK) return rc;
  if (n->rows == 0) {
    if (dgamma) MOE_CUDA_CHECK(cudaMemsetAsync(dgamma, 0, size_t(n->cols) * 4, stream));
    if (dbeta) MOE_CUDA_CHECK(cudaMemsetAsync(dbeta, 0, size_t(n->cols) * 4, stream));
    return MOE_OK;
  }
  if (!dy || !h || !gamma || !mean || !rstd || !dx) return MOE_ERR_INVALID_ARG;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < norm_ws_bytes(*n))
    return MOE_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  return n->dtype == MOE_F32
             ? norm_backward_t<float>(*n, dy, h, gamma, mean, rstd, dh, dx, dgamma, dbeta, w, stream)
             : norm_backward_t<__nv_bfloat16>(*n, dy, h, gamma, mean, rstd, dh, dx, dgamma, dbeta, w,
                                              stream);
}

}  // extern "C"
