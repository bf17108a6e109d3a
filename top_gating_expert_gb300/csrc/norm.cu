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
// Ring kernels (norm_fwd_ring_kernel, norm_bwd_ring_kernel), for many rows: CTAs of 16 warps, one an
// SM, L lanes a row (by its length, from one lane to 16 warps) and 512 / L rows at a time, each
// group of lanes walking rows of its own. A lane copies its own pieces of the rows to come into its own shared memory with
// cp.async and reads only those back, so the copies need no barrier; 64 to 128 KB an SM are
// then in flight whatever the registers hold. The two row sums of each direction cross the
// group's warps under a barrier of their own. gamma and beta stay in registers; the backward
// keeps the column sums of dgamma and dbeta there too (a column belongs to the same lane in
// every row), so dy and h are read once for all three results. The CTAs' partial sums are added
// by norm_bwd_sum_kernel in CTA order.
// Rows on no 16-byte boundary: norm_odd.cu. norm_fwd_kernel, in registers without the ring, is for few
// rows (one vector a lane, more warps a row: latency). Rows too long for any of these take the *_any
// kernels, which walk a row again from cache.
//
// Measured (copy rate 6778 GB/s): 65536 x 1024 bf16 with residual and the sum stored, 537 MB, 95 us
// (0.83 of it; without the ring 109 us); 16384 x 4096 bf16 backward with dh, 537 MB, 101 us (0.78;
// 250 us in registers alone, one row of 16 warps at a time, bound by its latency; now 72 % of the
// issue slots are taken); 65536 x 64 forward 6.6 us, backward 10 us (21 and 24 with a warp a row).
#include <algorithm>

#include "norm_ring.cuh"

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

// dgamma (blockIdx.y 0) and dbeta (1) from the slices' partials [slices][2][cols].
__global__ void __launch_bounds__(1024)
    norm_bwd_sum_kernel(const float* __restrict__ part, int slices, int cols, float* dgamma,
                        float* dbeta) {
  __shared__ float s_part[32][33];
  pdl_wait();
  pdl_trigger();
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  column_sums(slices, blockIdx.x * 32, cols, s_part,
              [&](int s, int c) { return part[(int64_t(s) * 2 + blockIdx.y) * cols + c]; },
              [&](int c, float t) { out[c] = t; });
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
  float t = s_red[warp / G * G + (threadIdx.x & (G - 1))];
  for (int off = G >> 1; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
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

// ------------------------------------------------------------------ ring kernels
template <typename T, int VEC, int NV, bool SUB = false>
__global__ void __launch_bounds__(32 * kRingWarps, 1)
    norm_fwd_ring_kernel(const T* x, const T* res, const float* __restrict__ gamma,
                         const float* __restrict__ beta, T* h, T* y, float* mean, float* rstd, int L,
                         moe_norm_t n) {
  constexpr int BYTES = VEC * int(sizeof(T));
  extern __shared__ __align__(16) uint8_t s_ring[];  // [stage][stream][NV][thread] pieces
  __shared__ float s_red[kRingWarps / 2][2][kRingWarps];  // rows of two warps or more
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const int slots = 32 * kRingWarps / L, slot = tid / L, rl = tid & (L - 1);
  const int M = n.cols, step = L * VEC, c0 = rl * VEC;
  float(*red)[kRingWarps] = s_red[L > 32 ? slot : 0];
  const int streams = res ? 2 : 1;
  auto piece = [&](int stage, int stream, int i) {
    return s_ring + size_t(((stage * streams + stream) * NV + i) * (32 * kRingWarps) + tid) * BYTES;
  };
  float g[NV][VEC], b[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) g[i][q] = b[i][q] = 0.f;
    if (c0 + i * step < M) {
      load_floats<VEC>(gamma + c0 + i * step, g[i]);
      if (beta) load_floats<VEC>(beta + c0 + i * step, b[i]);
    }
  }
  const int64_t stride = int64_t(gridDim.x) * slots;
  auto fetch = [&](int64_t r, int stage) {
    if (r < n.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * step;
        if (c < M) {
          copy_async(piece(stage, 0, i), x + r * n.ldx + c);
          if (res) copy_async(piece(stage, 1, i), res + r * n.ldr + c);
        }
      }
    }
    copy_commit();  // an empty group at the end: the waits count groups
  };
  int64_t r = int64_t(blockIdx.x) * slots + slot;
#pragma unroll
  for (int s = 0; s < kFwdStages - 1; ++s) fetch(r + s * stride, s);
  int stage = 0;
  // (a warp of several rows goes on while any of them exists; first: its lowest)
  const int first = SUB ? (tid & 31) / L : 0;
  for (; r - first < n.rows; r += stride) {
    const bool on = !SUB || r < n.rows;
    fetch(r + (kFwdStages - 1) * stride, stage == 0 ? kFwdStages - 1 : stage - 1);
    copy_wait<kFwdStages - 1>();
    float v[NV][VEC], s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
#pragma unroll
      for (int q = 0; q < VEC; ++q) v[i][q] = 0.f;
      if (on && c < M) {
        const Vec<T, VEC> xv = load_piece<T, VEC>(piece(stage, 0, i));
#pragma unroll
        for (int q = 0; q < VEC; ++q) v[i][q] = to_f32(xv.v[q]);
        if (res) {
          const Vec<T, VEC> rv = load_piece<T, VEC>(piece(stage, 1, i));
#pragma unroll
          for (int q = 0; q < VEC; ++q) v[i][q] += to_f32(rv.v[q]);
        }
        if (h) {
          Vec<T, VEC> o;
#pragma unroll
          for (int q = 0; q < VEC; ++q) o.v[q] = from_f32<T>(v[i][q]);
          store_vec<T, VEC>(h + r * n.ldh + c, o);
        }
      }
#pragma unroll
      for (int q = 0; q < VEC; ++q) s += v[i][q];
    }
    stage = stage + 1 == kFwdStages ? 0 : stage + 1;
    const float mu = row_lanes_sum<SUB>(s, L, slot, red[0]) / float(M);
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
    const float rs = 1.f / sqrtf(row_lanes_sum<SUB>(ss, L, slot, red[1]) / float(M) + n.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
      if (!on || c >= M) continue;
      Vec<T, VEC> o;
#pragma unroll
      for (int q = 0; q < VEC; ++q) o.v[q] = from_f32<T>(fmaf(v[i][q] * rs, g[i][q], b[i][q]));
      store_vec<T, VEC>(y + r * n.ldy + c, o);
    }
    if (on && rl == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
  }
}

// part: [gridDim.x][2][cols], null when neither dgamma nor dbeta is wanted.
template <typename T, int VEC, int NV, int STAGES, bool SUB = false>
__global__ void __launch_bounds__(32 * kRingWarps, 1)
    norm_bwd_ring_kernel(const T* dy, const T* h, const float* __restrict__ gamma,
                         const float* __restrict__ mean, const float* __restrict__ rstd, const T* dh, T* dx,
                         float* __restrict__ part, int L, moe_norm_t n) {
  constexpr int BYTES = VEC * int(sizeof(T));
  extern __shared__ __align__(16) uint8_t s_ring[];  // [stage][stream][NV][thread] pieces, then
                                                     // the slots' column sums
  __shared__ float s_red[kRingWarps / 2][4][kRingWarps];  // rows of two warps or more
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  const int slots = 32 * kRingWarps / L, slot = tid / L;
  const int M = n.cols, step = L * VEC, c0 = (tid & (L - 1)) * VEC, G = L >> 5;
  const int streams = dh ? 3 : 2;
  const float inv_m = 1.f / float(M);
  auto piece = [&](int stage, int stream, int i) {
    return s_ring + size_t(((stage * streams + stream) * NV + i) * (32 * kRingWarps) + tid) * BYTES;
  };
  float g[NV][VEC], sg[NV][VEC], sb[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int q = 0; q < VEC; ++q) g[i][q] = sg[i][q] = sb[i][q] = 0.f;
    if (c0 + i * step < M) load_floats<VEC>(gamma + c0 + i * step, g[i]);
  }
  const int64_t stride = int64_t(gridDim.x) * slots;
  auto fetch = [&](int64_t r, int stage) {
    if (r < n.rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * step;
        if (c < M) {
          copy_async(piece(stage, 0, i), h + r * n.ldx + c);
          copy_async(piece(stage, 1, i), dy + r * n.ldy + c);
          if (dh) copy_async(piece(stage, 2, i), dh + r * n.ldr + c);
        }
      }
    }
    copy_commit();
  };
  int64_t r = int64_t(blockIdx.x) * slots + slot;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(r + s * stride, s);
  float mu = r < n.rows ? __ldg(mean + r) : 0.f, rs = r < n.rows ? __ldg(rstd + r) : 0.f;
  int stage = 0, odd = 0;
  const int first = SUB ? lane / L : 0;  // (as in the forward)
  for (; r - first < n.rows; r += stride) {
    const bool on = !SUB || r < n.rows;
    fetch(r + (STAGES - 1) * stride, stage == 0 ? STAGES - 1 : stage - 1);
    const float mu_r = mu, rs_r = rs;
    if (r + stride < n.rows) {
      mu = __ldg(mean + r + stride);
      rs = __ldg(rstd + r + stride);
    }
    copy_wait<STAGES - 1>();
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!on || c0 + i * step >= M) continue;
      const Vec<T, VEC> hv = load_piece<T, VEC>(piece(stage, 0, i)), dv = load_piece<T, VEC>(piece(stage, 1, i));
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        const float d = to_f32(dv.v[q]), xh = __fmul_rn(to_f32(hv.v[q]) - mu_r, rs_r);
        const float gd = product(d, g[i][q]);
        sg[i][q] = fmaf(d, xh, sg[i][q]);
        sb[i][q] += d;
        s1 += gd;
        s2 = fmaf(gd, xh, s2);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      if (SUB && off >= L) continue;
      s1 += __shfl_xor_sync(0xffffffffu, s1, off);
      s2 += __shfl_xor_sync(0xffffffffu, s2, off);
    }
    if (!SUB && G > 1) {
      float* red = s_red[slot][2 * odd];  // two places in turn: one barrier a row
      if (lane == 0) {
        red[(tid >> 5) & (G - 1)] = s1;
        red[kRingWarps + ((tid >> 5) & (G - 1))] = s2;
      }
      asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(L) : "memory");
      s1 = red[lane & (G - 1)];
      s2 = red[kRingWarps + (lane & (G - 1))];
      for (int off = G >> 1; off > 0; off >>= 1) {
        s1 += __shfl_xor_sync(0xffffffffu, s1, off);
        s2 += __shfl_xor_sync(0xffffffffu, s2, off);
      }
    }
    s1 *= inv_m;
    s2 *= inv_m;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = c0 + i * step;
      if (!on || c >= M) continue;
      const Vec<T, VEC> hv = load_piece<T, VEC>(piece(stage, 0, i)), dv = load_piece<T, VEC>(piece(stage, 1, i));
      Vec<T, VEC> ev, o;
      if (dh) ev = load_piece<T, VEC>(piece(stage, 2, i));
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        const float xh = __fmul_rn(to_f32(hv.v[q]) - mu_r, rs_r);
        float v = rs_r * (product(to_f32(dv.v[q]), g[i][q]) - s1 - xh * s2);
        if (dh) v += to_f32(ev.v[q]);
        o.v[q] = from_f32<T>(v);
      }
      store_vec<T, VEC>(dx + r * n.ldh + c, o);
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    odd ^= 1;
  }
  if (!part) return;
  // the slots' column sums, added in slot order (several rows a warp: first across the warp)
  copy_wait<0>();
  if constexpr (SUB) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < VEC; ++q)
        for (int off = 16; off >= L; off >>= 1) {
          sg[i][q] += __shfl_xor_sync(0xffffffffu, sg[i][q], off);
          sb[i][q] += __shfl_xor_sync(0xffffffffu, sb[i][q], off);
        }
  }
  float* s_cols = reinterpret_cast<float*>(s_ring);
  const int width = step * NV, parts = min(slots, kRingWarps), mine = SUB ? tid >> 5 : slot;
  float* out = part + int64_t(blockIdx.x) * 2 * M;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    if (!SUB || lane < L) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < VEC; ++q) s_cols[mine * width + c0 + i * step + q] = which ? sb[i][q] : sg[i][q];
    }
    __syncthreads();
    for (int c = tid; c < M; c += 32 * kRingWarps) {
      float t = 0.f;
      for (int w = 0; w < parts; ++w) t += s_cols[w * width + c];
      out[which * M + c] = t;
    }
  }
}

int check_norm(const moe_norm_t* n) {
  if (!n || n->rows < 0 || n->cols < 1 || !(n->eps >= 0.f) || n->eps > 3.0e38f) return MOE_ERR_INVALID_ARG;
  if (n->dtype != MOE_F32 && n->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  const int64_t M = n->cols;
  if (n->ldx < M || n->ldr < M || n->ldh < M || n->ldy < M) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// The ring kernels write a partial a CTA; the slices of rows that are not held whole share 2048 CTAs.
int any_slices(int cols) {
  return std::max(1, std::min(kMaxPartials, 2048 / ((cols + kSliceCols - 1) / kSliceCols)));
}
size_t norm_ws_bytes(const moe_norm_t& n) {
  return 256 + align256(size_t(kMaxPartials) * 2 * size_t(n.cols) * 4);
}

bool vec_ok(const void* p, int64_t ld, int vec, size_t eb) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % vec == 0 && eb * vec == 16);
}

template <typename T, int VEC>
int norm_forward_v(const moe_norm_t& n, const T* x, const T* res, const float* gamma, const float* beta,
                   T* h, T* y, float* mean, float* rstd, cudaStream_t st) {
  // vectors a lane: one while the rows are few (more warps share a row's latency), else up to
  // 32 floats a lane
  constexpr int kMost = VEC == 8 ? 4 : 8;
  const bool few = n.rows <= 2 * num_sms();
  if constexpr (VEC == 1) {
    if ((!few || !row_warps(n.cols, VEC, kMost)) && norm_odd_fits<T>(n.cols))
      return norm_forward_odd<T>(n, x, res, gamma, beta, h, y, mean, rstd, st);
  } else {
    constexpr int kRing = 4;  // what shared memory holds
    int nv = 1;
    int G = row_warps(n.cols, VEC, nv, 1);
    while (G == 0 && nv < kRing) G = row_warps(n.cols, VEC, nv *= 2, nv == kRing ? 16 : 1);
    if (G) spread_rows(n.rows, nv, G);
    if (!few && G) {
      const int L = row_lanes(n.cols, VEC, nv, G), slots = 32 * kRingWarps / L;
      const unsigned grid = unsigned(std::min<int64_t>((n.rows + slots - 1) / slots, num_sms()));
      const size_t smem = size_t(kFwdStages) * (res ? 2 : 1) * nv * 32 * kRingWarps * VEC * sizeof(T);
      const size_t most = size_t(kFwdStages) * 2 * nv * 32 * kRingWarps * VEC * sizeof(T);
      auto go = [&](auto kern, auto) -> int {
        static std::atomic<unsigned long long> seen{0};
        if (const int rc = allow_smem(reinterpret_cast<const void*>(kern), int(most), seen)) return rc;
        return launch_kernel(kern, dim3(grid), dim3(32 * kRingWarps), smem, st, x, res, gamma, beta, h, y, mean,
                             rstd, L, n);
      };
      switch (nv) {
        case 1: return L < 32 ? go(norm_fwd_ring_kernel<T, VEC, 1, true>, Tag<0>{})
                              : go(norm_fwd_ring_kernel<T, VEC, 1>, Tag<1>{});
        case 2: return go(norm_fwd_ring_kernel<T, VEC, 2>, Tag<2>{});
        case 4: return go(norm_fwd_ring_kernel<T, VEC, 4>, Tag<4>{});
      }
    }
  }
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
  return launch_kernel(norm_bwd_sum_kernel, dim3(unsigned((cols + 31) / 32), 2), dim3(1024), 0, st, part,
                       slices, cols, dgamma, dbeta);
}

// CTAs that wrote a partial to part: *slices
template <typename T>
int norm_backward_ring(const moe_norm_t& n, const T* dy, const T* h, const float* gamma, const float* mean,
                       const float* rstd, const T* dh, T* dx, float* part, int nv, int G, int* slices,
                       cudaStream_t st) {
  constexpr int VEC = 16 / int(sizeof(T));
  const int L = row_lanes(n.cols, VEC, nv, G), slots = 32 * kRingWarps / L;
  const int grid = int(std::min<int64_t>((n.rows + slots - 1) / slots, std::min(num_sms(), kMaxPartials)));
  *slices = grid;
  auto go = [&](auto kern, int stages, auto) -> int {
    const size_t ring = size_t(stages) * (dh ? 3 : 2) * nv * 32 * kRingWarps * VEC * sizeof(T);
    const size_t cols = size_t(kRingWarps) * 32 * VEC * nv * 4;
    const size_t smem = std::max(ring, part ? cols : size_t(0));
    const size_t most = std::max(size_t(stages) * 3 * nv * 32 * kRingWarps * VEC * sizeof(T), cols);
    static std::atomic<unsigned long long> seen{0};
    if (const int rc = allow_smem(reinterpret_cast<const void*>(kern), int(most), seen)) return rc;
    return launch_kernel(kern, dim3(unsigned(grid)), dim3(32 * kRingWarps), smem, st, dy, h, gamma, mean, rstd,
                         dh, dx, part, L, n);
  };
  switch (nv) {
    case 1: return L < 32 ? go(norm_bwd_ring_kernel<T, VEC, 1, 3, true>, 3, Tag<0>{})
                          : go(norm_bwd_ring_kernel<T, VEC, 1, 3>, 3, Tag<1>{});
    case 2: return go(norm_bwd_ring_kernel<T, VEC, 2, 3>, 3, Tag<2>{});
  }
  return go(norm_bwd_ring_kernel<T, VEC, 4, 2>, 2, Tag<4>{});
}

template <typename T, bool ALIGNED>
int norm_backward_v(const moe_norm_t& n, const T* dy, const T* h, const float* gamma, const float* mean,
                    const float* rstd, const T* dh, T* dx, float* dgamma, float* dbeta, float* part,
                    cudaStream_t st) {
  constexpr int VEC = 16 / int(sizeof(T));
  int rc, slices = 0;
  const bool sums = dgamma || dbeta;
  // more vectors a lane before more warps a row, up to 16 columns a lane (32 column sums and 16 of
  // gamma: no spills); twice that for the longest bf16 rows (for fp32 vectors shared memory does not
  // hold it). Three stages, two where they would not fit
  constexpr int kMore = VEC == 8 ? 2 : 4;
  int nv = 1;
  int G = row_warps(n.cols, VEC, nv, 1);
  while (G == 0 && nv < 4) G = row_warps(n.cols, VEC, nv *= 2, nv >= kMore ? 16 : 1);
  if (G) {
    float* const to = sums ? part : nullptr;
    if constexpr (ALIGNED)
      rc = norm_backward_ring<T>(n, dy, h, gamma, mean, rstd, dh, dx, to, nv, G, &slices, st);
    else
      rc = norm_backward_odd<T>(n, dy, h, gamma, mean, rstd, dh, dx, to, nv, G, &slices, st);
    if (rc != MOE_OK || !sums) return rc;
    return launch_norm_sum(part, slices, n.cols, dgamma, dbeta, st);
  }
  // too long for the registers: the column sums first (dx may be written over dy)
  if (sums) {
    const int cblocks = (n.cols + kSliceCols - 1) / kSliceCols;
    slices = std::min(any_slices(n.cols), (n.rows + kWarpsN - 1) / kWarpsN);
    const int slice = (n.rows + slices - 1) / slices;
    slices = (n.rows + slice - 1) / slice;
    if ((rc = launch_kernel(norm_bwd_cols_any_kernel<T>, dim3(unsigned(cblocks), unsigned(slices)),
                            dim3(kThreadsN), 0, st, dy, h, mean, rstd, part, slice, n)) != MOE_OK)
      return rc;
    if ((rc = launch_norm_sum(part, slices, n.cols, dgamma, dbeta, st)) != MOE_OK) return rc;
  }
  return launch_kernel(norm_bwd_dx_any_kernel<T>, dim3(unsigned(n.rows)), dim3(kThreadsN), 0, st, dy, h, gamma,
                       mean, rstd, dh, dx, n);
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
  return vec ? norm_backward_v<T, true>(n, dyt, ht, gamma, mean, rstd, dht, dxt, dgamma, dbeta, part, st)
             : norm_backward_v<T, false>(n, dyt, ht, gamma, mean, rstd, dht, dxt, dgamma, dbeta, part, st);
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
