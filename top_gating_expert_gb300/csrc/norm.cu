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
//
// norm_fwd_kernel, norm_bwd_kernel: G warps a row (G = 1 .. 16, by the row's length), each lane NV
// 16-byte vectors of it, held in registers from the one load to the store; the two row sums of
// each direction cross the warps through shared memory. The backward's CTAs walk rows and keep
// the column sums of dgamma and dbeta in registers, a column belonging to the same lane in
// every row, so dy and h are read once for all three results; the CTAs' partial sums are
// added by norm_bwd_sum_kernel in CTA order. Rows that no 16-byte access fits take the same
// kernels with one element a vector. Rows too long for the registers take the *_any kernels,
// which walk a row again from cache.
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

// dgamma and dbeta from the slices' partials [slices][2][cols]: a CTA takes 32 columns of one of
// the two, each of its eight warps every eighth slice, then the warps' sums in order.
__global__ void __launch_bounds__(kThreadsN)
    norm_bwd_sum_kernel(const float* __restrict__ part, int slices, int cols, float* dgamma,
                        float* dbeta) {
  __shared__ float s_part[kWarpsN][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  float t = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int s = warp; s < slices; s += kWarpsN) t += part[(int64_t(s) * 2 + blockIdx.y) * cols + c];
  }
  s_part[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && c < cols) {
    for (int w = 1; w < kWarpsN; ++w) t += s_part[w][lane];
    out[c] = t;
  }
}

// Sum over the G warps of each row (warp = slot * G + wi), a fixed tree; every lane gets it.
// s_red: one float a warp, not written again before another barrier.
__device__ __forceinline__ float row_sum(float v, int G, float* s_red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (G == 1) return v;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) s_red[warp] = v;
  __syncthreads();
  const float* r = s_red + warp / G * G;
  float t = 0.f;
  for (int w = 0; w < G; ++w) t += r[w];
  return t;
}

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(512)
    norm_fwd_kernel(const T* x, const T* res, const float* __restrict__ gamma, const float* __restrict__ beta,
                    T* h, T* y, float* mean, float* rstd, int G, moe_norm_t n) {
  __shared__ float s_red[2][16];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slots = (blockDim.x >> 5) / G;
  const int64_t r = int64_t(blockIdx.x) * slots + warp / G;
  const int M = n.cols, step = G * 32 * VEC;
  const int c0 = (warp % G * 32 + lane) * VEC;
  const bool on = r < n.rows;
  float v[NV][VEC];
  float s = 0.f;
  {
    Vec<T, VEC> xv[NV], rv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
      if (on && c < M) {
        xv[i] = load_vec<T, VEC>(x + r * n.ldx + c);
        if (res) rv[i] = load_vec<T, VEC>(res + r * n.ldr + c);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        v[i][q] = 0.f;
        if (on && c < M) v[i][q] = to_f32(xv[i].v[q]) + (res ? to_f32(rv[i].v[q]) : 0.f);
        s += v[i][q];
      }
      if (h && on && c < M) {
        Vec<T, VEC> o;
#pragma unroll
        for (int q = 0; q < VEC; ++q) o.v[q] = from_f32<T>(v[i][q]);
        store_vec<T, VEC>(h + r * n.ldh + c, o);
      }
    }
  }
  const float mu = row_sum(s, G, s_red[0]) / float(M);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (c0 + i * step < M) {
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        v[i][q] -= mu;
        ss = fmaf(v[i][q], v[i][q], ss);
      }
    }
  const float rs = 1.f / sqrtf(row_sum(ss, G, s_red[1]) / float(M) + n.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = c0 + i * step;
    if (!on || c >= M) continue;
    float g[VEC], b[VEC];
    load_floats<VEC>(gamma + c, g);
    if (beta) load_floats<VEC>(beta + c, b);
    Vec<T, VEC> o;
#pragma unroll
    for (int q = 0; q < VEC; ++q) o.v[q] = from_f32<T>(fmaf(v[i][q] * rs, g[q], beta ? b[q] : 0.f));
    store_vec<T, VEC>(y + r * n.ldy + c, o);
  }
  if (on && lane == 0 && warp % G == 0) {
    if (mean) mean[r] = mu;
    if (rstd) rstd[r] = rs;
  }
}

// part: [gridDim.x][2][cols], null when neither dgamma nor dbeta is wanted.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(512)
    norm_bwd_kernel(const T* dy, const T* __restrict__ h, const float* __restrict__ gamma,
                    const float* __restrict__ mean, const float* __restrict__ rstd, const T* dh, T* dx,
                    float* __restrict__ part, int G, moe_norm_t n) {
  __shared__ float s_red[4][16];
  extern __shared__ float s_cols[];  // [slots][G * 32 * VEC * NV], one of the two sums at a time
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slots = (blockDim.x >> 5) / G, slot = warp / G;
  const int M = n.cols, step = G * 32 * VEC;
  const int c0 = (warp % G * 32 + lane) * VEC;
  const float inv_m = 1.f / float(M);
  float g[NV][VEC], sg[NV][VEC], sb[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) g[i][q] = sg[i][q] = sb[i][q] = 0.f;
    if (c0 + i * step < M) load_floats<VEC>(gamma + c0 + i * step, g[i]);
  }
  Vec<T, VEC> hv[NV], dv[NV];
  float mu = 0.f, rs = 0.f;
  auto fetch = [&](int64_t r) {
    if (r >= n.rows) return;
    mu = __ldg(mean + r);
    rs = __ldg(rstd + r);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
      if (c < M) {
        hv[i] = load_vec<T, VEC>(h + r * n.ldx + c);
        dv[i] = load_vec<T, VEC>(dy + r * n.ldy + c);
      }
    }
  };
  const int64_t stride = int64_t(gridDim.x) * slots;
  int64_t r = int64_t(blockIdx.x) * slots + slot;
  fetch(r);
  int buf = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * slots; r0 < n.rows; r0 += stride, r += stride, buf ^= 2) {
    const bool on = r < n.rows;
    const float rstd_r = rs;
    float xh[NV][VEC], gd[NV][VEC];
    Vec<T, VEC> ev[NV];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
      if (on && c < M) {
        if (dh) ev[i] = load_vec<T, VEC>(dh + r * n.ldr + c);
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
          const float d = to_f32(dv[i].v[q]);
          xh[i][q] = (to_f32(hv[i].v[q]) - mu) * rs;
          gd[i][q] = product(d, g[i][q]);
          sg[i][q] = fmaf(d, xh[i][q], sg[i][q]);
          sb[i][q] += d;
          s1 += gd[i][q];
          s2 = fmaf(gd[i][q], xh[i][q], s2);
        }
      }
    }
    fetch(r + stride);  // the next row, while this one's sums cross the warps
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      s1 += __shfl_xor_sync(0xffffffffu, s1, off);
      s2 += __shfl_xor_sync(0xffffffffu, s2, off);
    }
    if (G > 1) {
      if (lane == 0) {
        s_red[buf][warp] = s1;
        s_red[buf + 1][warp] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.f;
      for (int w = 0; w < G; ++w) {
        s1 += s_red[buf][slot * G + w];
        s2 += s_red[buf + 1][slot * G + w];
      }
    }
    s1 *= inv_m;
    s2 *= inv_m;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
      if (on && c < M) {
        Vec<T, VEC> o;
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
          float v = rstd_r * (gd[i][q] - s1 - xh[i][q] * s2);
          if (dh) v += to_f32(ev[i].v[q]);
          o.v[q] = from_f32<T>(v);
        }
        store_vec<T, VEC>(dx + r * n.ldh + c, o);
      }
    }
  }
  if (!part) return;
  // the slots' column sums, added in slot order
  const int width = step * NV;
  float* out = part + int64_t(blockIdx.x) * 2 * M;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < VEC; ++q) s_cols[slot * width + c0 + i * step + q] = which ? sb[i][q] : sg[i][q];
    __syncthreads();
    for (int c = threadIdx.x; c < M; c += blockDim.x) {
      float t = 0.f;
      for (int w = 0; w < slots; ++w) t += s_cols[w * width + c];
      out[which * M + c] = t;
    }
  }
}

constexpr int kMaxSlices = 608;  // four CTAs an SM

int check_norm(const moe_norm_t* n) {
  if (!n || n->rows < 0 || n->cols < 1 || !(n->eps >= 0.f) || n->eps > 3.0e38f) return MOE_ERR_INVALID_ARG;
  if (n->dtype != MOE_F32 && n->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  const int64_t M = n->cols;
  if (n->ldx < M || n->ldr < M || n->ldh < M || n->ldy < M) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Rows held in registers are at most 8192 long; the slices of longer ones share 2048 CTAs.
int any_slices(int cols) { return std::max(1, std::min(kMaxSlices, 2048 / ((cols + kSliceCols - 1) / kSliceCols))); }
size_t norm_ws_bytes(const moe_norm_t& n) {
  const int slices = n.cols <= 8192 ? kMaxSlices : any_slices(n.cols);
  return 256 + align256(size_t(slices) * 2 * size_t(n.cols) * 4);
}

bool vec_ok(const void* p, int64_t ld, int vec, size_t eb) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % vec == 0 && eb * vec == 16);
}

// Warps a row (a power of two up to 16) so that NV vectors a lane hold it; 0: too long.
int row_warps(int cols, int vec, int nv) {
  int G = 1;
  while (G <= 16 && int64_t(G) * 32 * vec * nv < cols) G *= 2;
  return G <= 16 ? G : 0;
}

template <typename T, int VEC>
int norm_forward_v(const moe_norm_t& n, const T* x, const T* res, const float* gamma, const float* beta,
                   T* h, T* y, float* mean, float* rstd, cudaStream_t st) {
  // vectors a lane: one while the rows are few (more warps share a row's latency), else 32
  // floats a lane, which keeps more loads in flight per warp
  constexpr int kMost = VEC == 8 ? 4 : 8;
  const bool few = n.rows <= 2 * num_sms();
  int nv = few ? 1 : kMost;
  if (!few)  // no more than the row needs
    while (nv > 1 && 32 * VEC * (nv / 2) >= n.cols) nv /= 2;
  int G = row_warps(n.cols, VEC, nv);
  while (G == 0 && nv < kMost) G = row_warps(n.cols, VEC, nv *= 2);
  if (G == 0)
    return launch_kernel(norm_fwd_any_kernel<T>, dim3(unsigned(n.rows)), dim3(kThreadsN), 0, st, x, res,
                         gamma, beta, h, y, mean, rstd, n);
  const int warps = std::max(G, few ? 1 : 4), slots = warps / G;
  const dim3 grid(unsigned((n.rows + slots - 1) / slots)), block(unsigned(32 * warps));
  auto go = [&](auto kern) { return launch_kernel(kern, grid, block, 0, st, x, res, gamma, beta, h, y, mean, rstd, G, n); };
  switch (nv) {
    case 1: return go(norm_fwd_kernel<T, VEC, 1>);
    case 2: return go(norm_fwd_kernel<T, VEC, 2>);
    case 4: return go(norm_fwd_kernel<T, VEC, 4>);
  }
  if constexpr (kMost == 8) return go(norm_fwd_kernel<T, VEC, 8>);
  return MOE_ERR_UNSUPPORTED;
}

template <typename T>
int norm_forward_t(const moe_norm_t& n, const void* x, const void* residual, const float* gamma,
                   const float* beta, void* h, void* y, float* mean, float* rstd, cudaStream_t st) {
  constexpr int V = 16 / int(sizeof(T));
  const bool vec = n.cols % V == 0 && vec_ok(x, n.ldx, V, sizeof(T)) && vec_ok(residual, n.ldr, V, sizeof(T)) &&
                   vec_ok(h, n.ldh, V, sizeof(T)) && vec_ok(y, n.ldy, V, sizeof(T)) &&
                   reinterpret_cast<uintptr_t>(gamma) % 16 == 0 && reinterpret_cast<uintptr_t>(beta) % 16 == 0;
  const T *xt = static_cast<const T*>(x), *rt = static_cast<const T*>(residual);
  T *ht = static_cast<T*>(h), *yt = static_cast<T*>(y);
  return vec ? norm_forward_v<T, V>(n, xt, rt, gamma, beta, ht, yt, mean, rstd, st)
             : norm_forward_v<T, 1>(n, xt, rt, gamma, beta, ht, yt, mean, rstd, st);
}

int launch_norm_sum(const float* part, int slices, int cols, float* dgamma, float* dbeta, cudaStream_t st) {
  return launch_kernel(norm_bwd_sum_kernel, dim3(unsigned((cols + 31) / 32), 2), dim3(kThreadsN), 0, st, part,
                       slices, cols, dgamma, dbeta);
}

template <typename T, int VEC>
int norm_backward_v(const moe_norm_t& n, const T* dy, const T* h, const float* gamma, const float* mean,
                    const float* rstd, const T* dh, T* dx, float* dgamma, float* dbeta, float* part,
                    cudaStream_t st) {
  int rc;
  const bool sums = dgamma || dbeta;
  int nv = 1;
  constexpr int kMost = VEC == 1 ? 8 : 2;
  int G = row_warps(n.cols, VEC, nv);
  while (G == 0 && nv < kMost) G = row_warps(n.cols, VEC, nv *= 2);
  if (G == 0) {  // too long for the registers: the column sums first (dx may be written over dy)
    if (sums) {
      const int cblocks = (n.cols + kSliceCols - 1) / kSliceCols;
      int slices = std::min(any_slices(n.cols), (n.rows + kWarpsN - 1) / kWarpsN);
      const int slice = (n.rows + slices - 1) / slices;
      slices = (n.rows + slice - 1) / slice;
      if ((rc = launch_kernel(norm_bwd_cols_any_kernel<T>, dim3(unsigned(cblocks), unsigned(slices)),
                              dim3(kThreadsN), 0, st, dy, h, mean, rstd, part, slice, n)) != MOE_OK)
        return rc;
      if ((rc = launch_norm_sum(part, slices, n.cols, dgamma, dbeta, st)) != MOE_OK) return rc;
    }
    return launch_kernel(norm_bwd_dx_any_kernel<T>, dim3(unsigned(n.rows)), dim3(kThreadsN), 0, st, dy, h,
                         gamma, mean, rstd, dh, dx, n);
  }
  const int warps = std::max(G, 8), slots = warps / G;
  const int per_sm = 64 / warps > 4 ? 4 : (64 / warps > 2 ? 64 / warps : 2);
  const int64_t need = (int64_t(n.rows) + slots - 1) / slots;
  const int grid = int(std::min<int64_t>(need, std::min(kMaxSlices, per_sm * num_sms())));
  const size_t smem = sums ? size_t(warps) * 32 * VEC * nv * 4 : 0;
  auto go = [&](auto kern) -> int {
    MOE_CUDA_CHECK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
    return launch_kernel(kern, dim3(unsigned(grid)), dim3(unsigned(32 * warps)), smem, st, dy, h, gamma, mean, rstd,
                         dh, dx, sums ? part : nullptr, G, n);
  };
  rc = MOE_ERR_UNSUPPORTED;
  if (nv == 1) rc = go(norm_bwd_kernel<T, VEC, 1>);
  if (nv == 2) rc = go(norm_bwd_kernel<T, VEC, 2>);
  if constexpr (kMost == 8) {
    if (nv == 4) rc = go(norm_bwd_kernel<T, VEC, 4>);
    if (nv == 8) rc = go(norm_bwd_kernel<T, VEC, 8>);
  }
  if (rc != MOE_OK || !sums) return rc;
  return launch_norm_sum(part, grid, n.cols, dgamma, dbeta, st);
}

template <typename T>
int norm_backward_t(const moe_norm_t& n, const void* dy, const void* h, const float* gamma,
                    const float* mean, const float* rstd, const void* dh, void* dx, float* dgamma,
                    float* dbeta, char* ws, cudaStream_t st) {
  constexpr int V = 16 / int(sizeof(T));
  const bool vec = n.cols % V == 0 && vec_ok(dy, n.ldy, V, sizeof(T)) && vec_ok(h, n.ldx, V, sizeof(T)) &&
                   vec_ok(dh, n.ldr, V, sizeof(T)) && vec_ok(dx, n.ldh, V, sizeof(T)) &&
                   reinterpret_cast<uintptr_t>(gamma) % 16 == 0;
  const T *dyt = static_cast<const T*>(dy), *ht = static_cast<const T*>(h), *dht = static_cast<const T*>(dh);
  T* dxt = static_cast<T*>(dx);
  float* part = reinterpret_cast<float*>(ws + 256);
  return vec ? norm_backward_v<T, V>(n, dyt, ht, gamma, mean, rstd, dht, dxt, dgamma, dbeta, part, st)
             : norm_backward_v<T, 1>(n, dyt, ht, gamma, mean, rstd, dht, dxt, dgamma, dbeta, part, st);
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
