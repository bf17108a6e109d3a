// Layer norm, forward and backward, of rows that lie on no 16-byte boundary: odd lengths, odd
// strides, operands each on a boundary of their own. The mathematics, the lanes of a row and the
// ring of copies in flight are those of norm.cu's ring kernels.
//
// A row is split among units, a warp each (or the whole of a short row, several of them a warp): a
// unit's U lanes copy the aligned 16-byte pieces that hold its columns, one more than the columns
// fill, and read them back as 4-byte words, consecutive lanes consecutive words, from the row's
// offset into the first piece on: an fp32 column or a pair of bf16 columns, which for a row that
// begins on an odd bf16 element is cut out of two words. A lane keeps the same words of every row, so
// gamma, beta and the column sums stay in its registers, and the results leave as words the same
// way (to a row on an odd element the lanes pass on one half each; the unit's first and last element
// go alone). A copy ends with the row and is filled up with zeros; the piece in which a tensor
// begins is brought element by element, so that nothing outside of it is read.
//
// Measured (copy rate 6778 GB/s; in brackets one element a copy and a store): 65536 x 1003 fp32 forward
// 92 us (215), with residual and the sum stored 178 us, 5.9 TB/s (263), backward with dh 167 us, 6.3 TB/s
// (261); bf16 86 (162), 136 (204) and 146 us (277): half the bytes, as many
// instructions (64 and 72 % of the issue slots with four warps a scheduler). Pieces shifted in
// registers to 16 bytes of consecutive columns a lane, the results turned to words in shared memory,
// took 240 and 176 us for the two backwards.
#include <algorithm>

#include "norm_ring.cuh"

namespace moe {
namespace {

// 16 bytes, global to shared, of which `bytes` are read and the rest filled with zeros
__device__ __forceinline__ void copy_async_part(void* dst, const void* src, int bytes) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
}

// elements between the 16-byte boundary at or below p, and p
template <typename T>
__device__ __forceinline__ int lead_of(const T* p) {
  return int(reinterpret_cast<uintptr_t>(p) & 15) / int(sizeof(T));
}

// The piece that begins at element e0 of a row of M elements at `row` (of a tensor at `base`; on: the
// row exists). HEAD: e0 may be negative.
template <typename T, bool HEAD>
__device__ __forceinline__ void fetch_piece(uint4* to, const T* base, const T* row, int e0, int M, bool on) {
  constexpr int VEC = 16 / int(sizeof(T));
  const int here = on ? max(0, min(VEC, M - e0)) : 0;
  if (!HEAD || e0 >= 0 || here == 0 || row + e0 >= base) {
    copy_async_part(to, here ? row + e0 : base - lead_of(base), here * int(sizeof(T)));
  } else {  // the tensor begins inside this piece
    for (int q = -e0; q < VEC; ++q) reinterpret_cast<T*>(to)[q] = q < here ? row[e0 + q] : from_f32<T>(0.f);
  }
}

// A unit: its place, and the copies, reads and writes of its part of a row.
template <typename T, int NV>
struct Unit {
  static constexpr int VEC = 16 / int(sizeof(T)), EPW = 4 / int(sizeof(T)), NW = 4 * NV;
  int U, lu, u0, M, first_lane;  // lanes, this lane, first column, the row's length, lane of lu = 0
  __device__ __forceinline__ int col(int j) const { return u0 + EPW * (lu + U * j); }

  __device__ __forceinline__ void fetch(uint4* to, const T* base, int64_t ld, int64_t r, bool on) const {
    const T* row = base + (on ? r : 0) * ld;
    const int e0 = u0 - lead_of(row) + VEC * lu;
    fetch_piece<T, true>(to + lu, base, row, e0, M, on);
#pragma unroll
    for (int i = 1; i < NV; ++i) fetch_piece<T, false>(to + i * U + lu, base, row, e0 + VEC * U * i, M, on);
    if (lu == U - 1) fetch_piece<T, false>(to + NV * U, base, row, e0 + VEC * (U * (NV - 1) + 1), M, on);
  }
  // this lane's words of the row that starts at `row`; zeros beyond its end
  __device__ __forceinline__ void take(const uint4* from, const T* row, uint32_t (&w)[NW]) const {
    const int lead = lead_of(row);
    const uint32_t* p = reinterpret_cast<const uint32_t*>(from) + lead / EPW + lu;
    if (EPW == 2 && (lead & 1)) {
#pragma unroll
      for (int j = 0; j < NW; ++j) w[j] = __funnelshift_r(p[U * j], p[U * j + 1], 16);
    } else {
#pragma unroll
      for (int j = 0; j < NW; ++j) w[j] = p[U * j];
    }
  }
  // the words to a row (all lanes of the warp; on: the row exists)
  __device__ __forceinline__ void put(T* row, const uint32_t (&w)[NW], bool on) const {
    T* dst = row + u0;
    const int count = on ? max(0, min(EPW * U * NW, M - u0)) : 0;
    if constexpr (EPW == 1) {
#pragma unroll
      for (int j = 0; j < NW; ++j)
        if (lu + U * j < count) reinterpret_cast<uint32_t*>(dst)[lu + U * j] = w[j];
    } else {
      const int odd = int(reinterpret_cast<uintptr_t>(dst) >> 1) & 1;
      const int words = (count - odd) >> 1;
      const bool rest = count > odd && ((count - odd) & 1);  // an element beyond the last whole word
      uint32_t* out = reinterpret_cast<uint32_t*>(dst + odd);
      if (__any_sync(0xffffffffu, odd)) {
        const int from = first_lane + ((lu + 1) & (U - 1));
#pragma unroll
        for (int j = 0; j < NW; ++j) {
          // the next word: of the lane beside, the last lane's next one of the first lane
          const uint32_t mine = lu == 0 && j + 1 < NW ? w[j + 1 < NW ? j + 1 : j] : w[j];
          const uint32_t next = __shfl_sync(0xffffffffu, mine, from);
          const uint32_t v = __funnelshift_r(w[j], next, 16 * odd);
          const int k = lu + U * j;
          if (k < words) out[k] = v;
          else if (rest && k == words)
            reinterpret_cast<uint16_t*>(dst)[count - 1] = uint16_t(odd ? w[j] >> 16 : w[j]);
        }
        if (lu == 0 && odd && count > 0) reinterpret_cast<uint16_t*>(dst)[0] = uint16_t(w[0]);
      } else {
#pragma unroll
        for (int j = 0; j < NW; ++j) {
          const int k = lu + U * j;
          if (k < words) out[k] = w[j];
          else if (rest && k == words) reinterpret_cast<uint16_t*>(dst)[count - 1] = uint16_t(w[j]);
        }
      }
    }
  }
  static __device__ __forceinline__ float value(uint32_t w, int e) {
    if constexpr (EPW == 1) return __uint_as_float(w);
    else return __uint_as_float(e ? w & 0xffff0000u : w << 16);
  }
  static __device__ __forceinline__ uint32_t word(const float (&v)[EPW]) {
    if constexpr (EPW == 1) {
      return __float_as_uint(v[0]);
    } else {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[0], v[EPW - 1]);
      return *reinterpret_cast<const uint32_t*>(&p);
    }
  }
};

template <typename T, int NV, bool SUB>
__global__ void __launch_bounds__(32 * kRingWarps, 1)
    norm_fwd_odd_kernel(const T* x, const T* res, const float* __restrict__ gamma,
                        const float* __restrict__ beta, T* h, T* y, float* mean, float* rstd, int L,
                        moe_norm_t n) {
  using Un = Unit<T, NV>;
  constexpr int EPW = Un::EPW, NW = Un::NW, THREADS = 32 * kRingWarps;
  extern __shared__ __align__(16) uint4 s_odd[];  // [stage][stream][unit][U NV + 1] pieces
  __shared__ float s_red[kRingWarps / 2][2][kRingWarps];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, slots = THREADS / L, slot = tid / L, rl = tid & (L - 1);
  const int U = SUB ? L : 32, unit = tid / U, M = n.cols;
  const Un un{U, tid & (U - 1), rl / U * (U * NW * EPW), M, (tid & 31) & ~(U - 1)};
  float(*red)[kRingWarps] = s_red[L > 32 ? slot : 0];
  const int streams = res ? 2 : 1, per = THREADS * NV + THREADS / U;
  auto pieces = [&](int stage, int stream) { return s_odd + (stage * streams + stream) * per + unit * (U * NV + 1); };
  float g[NW][EPW], b[NW][EPW];
#pragma unroll
  for (int j = 0; j < NW; ++j)
#pragma unroll
    for (int e = 0; e < EPW; ++e) {
      const int c = un.col(j) + e;
      g[j][e] = c < M ? __ldg(gamma + c) : 0.f;
      b[j][e] = beta && c < M ? __ldg(beta + c) : 0.f;
    }
  const int64_t stride = int64_t(gridDim.x) * slots;
  auto fetch = [&](int64_t r, int stage) {
    un.fetch(pieces(stage, 0), x, n.ldx, r, r < n.rows);
    if (res) un.fetch(pieces(stage, 1), res, n.ldr, r, r < n.rows);
    copy_commit();
  };
  int64_t r = int64_t(blockIdx.x) * slots + slot;
#pragma unroll
  for (int s = 0; s < kFwdStages - 1; ++s) fetch(r + s * stride, s);
  int stage = 0;
  const int first = SUB ? (tid & 31) / L : 0;
  for (; r - first < n.rows; r += stride) {
    const bool on = !SUB || r < n.rows;
    __syncwarp();  // the unit's lanes have read the stage to be filled
    fetch(r + (kFwdStages - 1) * stride, stage == 0 ? kFwdStages - 1 : stage - 1);
    copy_wait<kFwdStages - 1>();
    __syncwarp();
    float v[NW][EPW], s = 0.f;
    {
      uint32_t w[NW];
      un.take(pieces(stage, 0), x + r * n.ldx, w);
#pragma unroll
      for (int j = 0; j < NW; ++j)
#pragma unroll
        for (int e = 0; e < EPW; ++e) v[j][e] = Un::value(w[j], e);
      if (res) {
        un.take(pieces(stage, 1), res + r * n.ldr, w);
#pragma unroll
        for (int j = 0; j < NW; ++j)
#pragma unroll
          for (int e = 0; e < EPW; ++e) v[j][e] += Un::value(w[j], e);
      }
      if (h) {
#pragma unroll
        for (int j = 0; j < NW; ++j) w[j] = Un::word(v[j]);
        un.put(h + r * n.ldh, w, on);
      }
    }
    stage = stage + 1 == kFwdStages ? 0 : stage + 1;
#pragma unroll
    for (int j = 0; j < NW; ++j)
#pragma unroll
      for (int e = 0; e < EPW; ++e) s += v[j][e];
    const float mu = row_lanes_sum<SUB>(s, L, slot, red[0]) / float(M);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NW; ++j)
#pragma unroll
      for (int e = 0; e < EPW; ++e) {
        v[j][e] = un.col(j) + e < M ? v[j][e] - mu : 0.f;
        ss = fmaf(v[j][e], v[j][e], ss);
      }
    const float rs = 1.f / sqrtf(row_lanes_sum<SUB>(ss, L, slot, red[1]) / float(M) + n.eps);
    uint32_t w[NW];
#pragma unroll
    for (int j = 0; j < NW; ++j) {
#pragma unroll
      for (int e = 0; e < EPW; ++e) v[j][e] = fmaf(v[j][e] * rs, g[j][e], b[j][e]);
      w[j] = Un::word(v[j]);
    }
    un.put(y + r * n.ldy, w, on);
    if (on && rl == 0) {
      if (mean) mean[r] = mu;
      if (rstd) rstd[r] = rs;
    }
  }
}

// part: [gridDim.x][2][cols], null when neither dgamma nor dbeta is wanted.
template <typename T, int NV, int STAGES, bool SUB>
__global__ void __launch_bounds__(32 * kRingWarps, 1)
    norm_bwd_odd_kernel(const T* dy, const T* h, const float* __restrict__ gamma,
                        const float* __restrict__ mean, const float* __restrict__ rstd, const T* dh, T* dx,
                        float* __restrict__ part, int L, moe_norm_t n) {
  using Un = Unit<T, NV>;
  constexpr int EPW = Un::EPW, NW = Un::NW, THREADS = 32 * kRingWarps;
  extern __shared__ __align__(16) uint4 s_odd[];  // (as in the forward), at last the column sums
  __shared__ float s_red[kRingWarps / 2][4][kRingWarps];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, slots = THREADS / L, slot = tid / L, G = L >> 5;
  const int U = SUB ? L : 32, unit = tid / U, M = n.cols;
  const Un un{U, tid & (U - 1), (tid & (L - 1)) / U * (U * NW * EPW), M, lane & ~(U - 1)};
  const int streams = dh ? 3 : 2, per = THREADS * NV + THREADS / U;
  const float inv_m = 1.f / float(M);
  auto pieces = [&](int stage, int stream) { return s_odd + (stage * streams + stream) * per + unit * (U * NV + 1); };
  float g[NW][EPW], sg[NW][EPW], sb[NW][EPW];
#pragma unroll
  for (int j = 0; j < NW; ++j)
#pragma unroll
    for (int e = 0; e < EPW; ++e) {
      const int c = un.col(j) + e;
      g[j][e] = c < M ? __ldg(gamma + c) : 0.f;
      sg[j][e] = sb[j][e] = 0.f;
    }
  const int64_t stride = int64_t(gridDim.x) * slots;
  auto fetch = [&](int64_t r, int stage) {
    un.fetch(pieces(stage, 0), h, n.ldx, r, r < n.rows);
    un.fetch(pieces(stage, 1), dy, n.ldy, r, r < n.rows);
    if (dh) un.fetch(pieces(stage, 2), dh, n.ldr, r, r < n.rows);
    copy_commit();
  };
  int64_t r = int64_t(blockIdx.x) * slots + slot;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(r + s * stride, s);
  float mu = r < n.rows ? __ldg(mean + r) : 0.f, rs = r < n.rows ? __ldg(rstd + r) : 0.f;
  int stage = 0, odd = 0;
  const int first = SUB ? lane / L : 0;
  for (; r - first < n.rows; r += stride) {
    const bool on = !SUB || r < n.rows;
    __syncwarp();
    fetch(r + (STAGES - 1) * stride, stage == 0 ? STAGES - 1 : stage - 1);
    const float mu_r = on ? mu : 0.f, rs_r = on ? rs : 0.f;  // (no row: nothing is added below)
    if (r + stride < n.rows) {
      mu = __ldg(mean + r + stride);
      rs = __ldg(rstd + r + stride);
    }
    copy_wait<STAGES - 1>();
    __syncwarp();
    float s1 = 0.f, s2 = 0.f;
    uint32_t hw[NW], dw[NW];
    un.take(pieces(stage, 0), h + r * n.ldx, hw);
    un.take(pieces(stage, 1), dy + r * n.ldy, dw);
#pragma unroll
    for (int j = 0; j < NW; ++j)  // beyond the row's end d = 0: nothing is added
#pragma unroll
      for (int e = 0; e < EPW; ++e) {
        const float d = Un::value(dw[j], e), xh = __fmul_rn(Un::value(hw[j], e) - mu_r, rs_r);
        const float gd = product(d, g[j][e]);
        sg[j][e] = fmaf(d, xh, sg[j][e]);
        sb[j][e] += d;
        s1 += gd;
        s2 = fmaf(gd, xh, s2);
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
    if constexpr (NW * EPW > 16) {  // the registers do not hold both: read again
      __syncwarp();
      un.take(pieces(stage, 0), h + r * n.ldx, hw);
      un.take(pieces(stage, 1), dy + r * n.ldy, dw);
    }
    uint32_t ew[NW];
    if (dh) un.take(pieces(stage, 2), dh + r * n.ldr, ew);
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      float o[EPW];
#pragma unroll
      for (int e = 0; e < EPW; ++e) {
        const float xh = __fmul_rn(Un::value(hw[j], e) - mu_r, rs_r);
        o[e] = rs_r * (product(Un::value(dw[j], e), g[j][e]) - s1 - xh * s2);
        if (dh) o[e] += Un::value(ew[j], e);
      }
      hw[j] = Un::word(o);
    }
    un.put(dx + r * n.ldh, hw, on);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    odd ^= 1;
  }
  if (!part) return;
  // the slots' column sums, added in slot order (several rows a warp: first across the warp)
  copy_wait<0>();
  if constexpr (SUB) {
#pragma unroll
    for (int j = 0; j < NW; ++j)
#pragma unroll
      for (int e = 0; e < EPW; ++e)
        for (int off = 16; off >= L; off >>= 1) {
          sg[j][e] += __shfl_xor_sync(0xffffffffu, sg[j][e], off);
          sb[j][e] += __shfl_xor_sync(0xffffffffu, sb[j][e], off);
        }
  }
  float* s_cols = reinterpret_cast<float*>(s_odd);
  const int width = L * NW * EPW, parts = min(slots, kRingWarps), mine = SUB ? tid >> 5 : slot;
  float* out = part + int64_t(blockIdx.x) * 2 * M;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    if (!SUB || lane < L) {
#pragma unroll
      for (int j = 0; j < NW; ++j)
#pragma unroll
        for (int e = 0; e < EPW; ++e) s_cols[mine * width + un.col(j) + e] = which ? sb[j][e] : sg[j][e];
    }
    __syncthreads();
    for (int c = tid; c < M; c += THREADS) {
      float t = 0.f;
      for (int w = 0; w < parts; ++w) t += s_cols[w * width + c];
      out[which * M + c] = t;
    }
  }
}

constexpr int kOddMost = 4;  // pieces a lane: what shared memory holds (of three streams, two stages)

// bytes of the ring
size_t odd_smem(int stages, int streams, int nv, int L) {
  const int threads = 32 * kRingWarps, U = std::min(L, 32);
  return size_t(16) * stages * streams * (threads * nv + threads / U);
}

}  // namespace

template <typename T>
bool norm_odd_fits(int cols) {
  return row_warps(cols, 16 / int(sizeof(T)), kOddMost) != 0;
}

template <typename T>
int norm_forward_odd(const moe_norm_t& n, const T* x, const T* res, const float* gamma, const float* beta, T* h,
                     T* y, float* mean, float* rstd, cudaStream_t st) {
  constexpr int VEC = 16 / int(sizeof(T));
  int nv = 1;
  int G = row_warps(n.cols, VEC, nv, 1);
  while (G == 0 && nv < kOddMost) G = row_warps(n.cols, VEC, nv *= 2, nv == kOddMost ? 16 : 1);
  spread_rows(n.rows, nv, G);
  const int L = row_lanes(n.cols, VEC, nv, G), slots = 32 * kRingWarps / L;
  const unsigned grid = unsigned(std::min<int64_t>((n.rows + slots - 1) / slots, num_sms()));
  const size_t smem = odd_smem(kFwdStages, res ? 2 : 1, nv, L);
  auto go = [&](auto kern, auto) -> int {
    static std::atomic<unsigned long long> seen{0};
    const size_t most = odd_smem(kFwdStages, 2, nv, nv == 1 ? 1 : 32);
    if (const int rc = allow_smem(reinterpret_cast<const void*>(kern), int(most), seen)) return rc;
    return launch_kernel(kern, dim3(grid), dim3(32 * kRingWarps), smem, st, x, res, gamma, beta, h, y, mean, rstd,
                         L, n);
  };
  switch (nv) {
    case 1: return L < 32 ? go(norm_fwd_odd_kernel<T, 1, true>, Tag<0>{})
                          : go(norm_fwd_odd_kernel<T, 1, false>, Tag<1>{});
    case 2: return go(norm_fwd_odd_kernel<T, 2, false>, Tag<2>{});
  }
  return go(norm_fwd_odd_kernel<T, 4, false>, Tag<4>{});
}

template <typename T>
int norm_backward_odd(const moe_norm_t& n, const T* dy, const T* h, const float* gamma, const float* mean,
                      const float* rstd, const T* dh, T* dx, float* part, int nv, int G, int* slices,
                      cudaStream_t st) {
  constexpr int VEC = 16 / int(sizeof(T));
  const int L = row_lanes(n.cols, VEC, nv, G), slots = 32 * kRingWarps / L;
  const int grid = int(std::min<int64_t>((n.rows + slots - 1) / slots, std::min(num_sms(), kMaxPartials)));
  *slices = grid;
  auto go = [&](auto kern, int stages, auto) -> int {
    const size_t cols = size_t(kRingWarps) * 32 * VEC * nv * 4;
    const size_t smem = std::max(odd_smem(stages, dh ? 3 : 2, nv, L), part ? cols : size_t(0));
    const size_t most = std::max(odd_smem(stages, 3, nv, nv == 1 ? 1 : 32), cols);
    static std::atomic<unsigned long long> seen{0};
    if (const int rc = allow_smem(reinterpret_cast<const void*>(kern), int(most), seen)) return rc;
    return launch_kernel(kern, dim3(unsigned(grid)), dim3(32 * kRingWarps), smem, st, dy, h, gamma, mean, rstd, dh,
                         dx, part, L, n);
  };
  switch (nv) {
    case 1: return L < 32 ? go(norm_bwd_odd_kernel<T, 1, 3, true>, 3, Tag<0>{})
                          : go(norm_bwd_odd_kernel<T, 1, 3, false>, 3, Tag<1>{});
    case 2: return go(norm_bwd_odd_kernel<T, 2, 3, false>, 3, Tag<2>{});
  }
  return go(norm_bwd_odd_kernel<T, 4, 2, false>, 2, Tag<4>{});
}

#define MOE_NORM_ODD(T)                                                                                          \
  template bool norm_odd_fits<T>(int);                                                                           \
  template int norm_forward_odd<T>(const moe_norm_t&, const T*, const T*, const float*, const float*, T*, T*,    \
                                   float*, float*, cudaStream_t);                                                \
  template int norm_backward_odd<T>(const moe_norm_t&, const T*, const T*, const float*, const float*,           \
                                    const float*, const T*, T*, float*, int, int, int*, cudaStream_t);
MOE_NORM_ODD(float)
MOE_NORM_ODD(__nv_bfloat16)
#undef MOE_NORM_ODD

}  // namespace moe
