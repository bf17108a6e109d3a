// The linear layer for one bf16 token, or up to eight fp32 ones (a serving step), on plain FMA.
//
// Bound by the read of W: every warp streams whole rows of it, contiguous along k, several loads in
// flight a lane, while x (all tokens' k range, fp32) sits in shared memory. The tensor-core tile
// reads 128 rows of W 128 bytes at a time on 112 of the 152 SMs (14336 x 4096: 27 us, here 19.4,
// 0.90 of the copy rate; 14335 x 4095, rows on no boundary, 23 us),
// and a matrix whose rows are on no 16-byte boundary would have to be copied first. From two bf16
// tokens on, the FMAs and the reads of x outweigh that (two tokens: 28 us here, 25 there). The first rows
// are asked for in L2 before the wait on the previous kernel, while x is staged.
//
// A CTA of 8 warps: `kw` warps share a row's k range (chosen so that the rows fill the GPU), the
// other factor is rows. fp32 sums; lanes and warps join in a fixed order.
#include <algorithm>
#include <type_traits>

#include "linear.cuh"

namespace moe {
namespace {

constexpr int kWarpsG = 8, kThreadsG = 32 * kWarpsG;
constexpr int kSliceK = 4096;  // x values of one token held at a time

struct FewArgs {
  const void* x;
  const void* W;
  int64_t ldx, ldw;
  int T, N, K, kw;
  LinearEpi e;
};

template <int VEC>
__device__ __forceinline__ void unpack(const uint4& w, float (&f)[VEC], std::integral_constant<int, 2>) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = __uint_as_float(u[q] << 16);
    f[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
  }
}
template <int VEC>
__device__ __forceinline__ void unpack(const uint4& w, float (&f)[VEC], std::integral_constant<int, 4>) {
  f[0] = __uint_as_float(w.x);
  f[1] = __uint_as_float(w.y);
  f[2] = __uint_as_float(w.z);
  f[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  return ld_nc_v4(static_cast<const uint4*>(p));
}

// acc[r][t] += over this slice's k of rows wr[r], in 16-byte pieces. SHIFT: rows on any element
// boundary (TT = 1): a row's first whole piece starts h elements in; the elements before it and
// after the last one are taken alone, and x is held in four copies, copy s with x[k] at k + s, of
// which the one with h + s a multiple of 4 gives 16-byte reads.
template <typename T, int TT, int R, bool SHIFT>
__device__ __forceinline__ void rows_vec(const T* (&wr)[R], const float* sx, int pitch, int len, int part, int parts,
                                         float (&acc)[R][TT]) {
  constexpr int VEC = 16 / int(sizeof(T)), U = 4;  // U pieces of each row in flight
  const int lane = threadIdx.x & 31;
  const T* w0[R];
  const float* xs[R];
  int nv[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    int h = 0;
    if constexpr (SHIFT) {
      h = (VEC - int((reinterpret_cast<uintptr_t>(wr[r]) & 15) / sizeof(T))) & (VEC - 1);
      if (h > len) h = len;
      if (part == 0) {
        const int tail = (len - h) % VEC;
        if (lane < h) acc[r][0] = fmaf(to_f32(wr[r][lane]), sx[lane], acc[r][0]);
        if (lane >= VEC && lane < VEC + tail) {
          const int k = len - tail + lane - VEC;
          acc[r][0] = fmaf(to_f32(wr[r][k]), sx[k], acc[r][0]);
        }
      }
    }
    w0[r] = wr[r] + h;
    const int s = (4 - (h & 3)) & 3;
    xs[r] = sx + s * pitch + s + h;
    nv[r] = (len - h) / VEC;
  }
  int most = nv[0];
#pragma unroll
  for (int r = 1; r < R; ++r) most = max(most, nv[r]);
  const int stride = 32 * parts;
  for (int i = part * 32 + lane; i < most; i += U * stride) {
    uint4 w[R][U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r)
        w[r][u] = i + u * stride < nv[r] ? ldg_stream(w0[r] + (i + u * stride) * VEC) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = i + u * stride;
      if (v >= most) break;
      float xv[TT][VEC];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (SHIFT && v >= nv[r]) continue;
        if (SHIFT || r == 0) {  // aligned rows share x
#pragma unroll
          for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int q = 0; q < VEC / 4; ++q)
              *reinterpret_cast<float4*>(&xv[t][4 * q]) =
                  *reinterpret_cast<const float4*>(xs[r] + t * pitch + v * VEC + 4 * q);
        }
        float f[VEC];
        unpack<VEC>(w[r][u], f, std::integral_constant<int, int(sizeof(T))>{});
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int q = 0; q < VEC; ++q) acc[r][t] = fmaf(f[q], xv[t][q], acc[r][t]);
      }
    }
  }
}

// fp32 rows of several tokens on any element boundary, an element at a time
template <int TT>
__device__ __forceinline__ void row_words(const float* wr, const float* sx, int slice, int len, int part, int parts,
                                          float (&acc)[TT]) {
  constexpr int U = 8;
  const int stride = 32 * parts;
  for (int i = part * 32 + (threadIdx.x & 31); i < len; i += U * stride) {
    float w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = i + u * stride < len ? __ldg(wr + i + u * stride) : 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u * stride >= len) break;
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[t] = fmaf(w[u], sx[t * slice + i + u * stride], acc[t]);
    }
  }
}

// floats of one token's (or one copy's) slice of x, with room for the shift
__host__ __device__ inline int few_pitch(int K) { return ((K < kSliceK ? K : kSliceK) + 3 + 3) / 4 * 4; }

template <typename T, int TT, bool VECTOR, int R>
__global__ void __launch_bounds__(kThreadsG) linear_few_kernel(FewArgs p) {
  constexpr bool SHIFT = !VECTOR && TT == 1;
  extern __shared__ __align__(16) float sx[];  // [TT or 4 copies][pitch] of x
  __shared__ float s_acc[kWarpsG][R][TT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pitch = few_pitch(p.K);
  const int part = warp % p.kw, rows_cta = kWarpsG / p.kw;
  const T* W = static_cast<const T*>(p.W);
  const T* x = static_cast<const T*>(p.x);
  if (part == 0 && lane < R) {  // the warp's first rows into L2 while the previous kernel ends
    const int64_t n = int64_t(blockIdx.x) * rows_cta * R + int64_t(warp / p.kw) * R + lane;
    if (n < p.N) {
      const uintptr_t a = (reinterpret_cast<uintptr_t>(W + n * p.ldw) + 15) & ~uintptr_t(15);
      const uintptr_t b = reinterpret_cast<uintptr_t>(W + n * p.ldw + p.K) & ~uintptr_t(15);
      if (a < b) prefetch_l2_bulk(reinterpret_cast<const void*>(a), uint32_t(min(b - a, uintptr_t(32768))));
    }
  }
  pdl_wait();
  pdl_trigger();
  const int64_t per = int64_t(gridDim.x) * rows_cta * R;
  for (int64_t n0 = (int64_t(blockIdx.x) * rows_cta) * R; n0 < p.N; n0 += per) {  // uniform over the CTA
    const int64_t n = n0 + int64_t(warp / p.kw) * R;
    float acc[R][TT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[r][t] = 0.f;
    for (int k0 = 0; k0 < p.K; k0 += kSliceK) {
      const int len = min(kSliceK, p.K - k0);
      if (p.K > kSliceK || n0 == int64_t(blockIdx.x) * rows_cta * R) {
        __syncthreads();
        for (int t = 0; t < TT; ++t)
          for (int k = tid; k < len; k += kThreadsG) {
            const float v = t < p.T ? to_f32(x[t * p.ldx + k0 + k]) : 0.f;
            sx[t * pitch + k] = v;
            if constexpr (SHIFT) {
#pragma unroll
              for (int s = 1; s < 4; ++s) sx[s * pitch + k + s] = v;
            }
          }
        __syncthreads();
      }
      if (n < p.N) {
        const T* wr[R];  // rows past the last repeat it; they are not stored
#pragma unroll
        for (int r = 0; r < R; ++r) wr[r] = W + min(n + r, int64_t(p.N) - 1) * p.ldw + k0;
        if constexpr (VECTOR || SHIFT) {
          rows_vec<T, TT, R, SHIFT>(wr, sx, pitch, len, part, p.kw, acc);
        } else {
#pragma unroll
          for (int r = 0; r < R; ++r) row_words<TT>(wr[r], sx, pitch, len, part, p.kw, acc[r]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], off);
    if (p.kw > 1) {
      if (lane == 0)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t = 0; t < TT; ++t) s_acc[warp][r][t] = acc[r][t];
      __syncthreads();
    }
    // lane (r, t) of the row's first warp finishes an output
    if (part == 0 && lane < R * TT) {
      const int r = lane / TT, t = lane % TT;
      float v = 0.f;
      if (p.kw > 1) {
        for (int w = 0; w < p.kw; ++w) v += s_acc[warp + w][r][t];
      } else {
#pragma unroll
        for (int rr = 0; rr < R; ++rr)
#pragma unroll
          for (int tt = 0; tt < TT; ++tt)
            if (rr == r && tt == t) v = acc[rr][tt];
      }
      const int64_t c = n + r;
      if (c < p.N && t < p.T) {
        if (p.e.bias) v += p.e.bias[c];
        if (p.e.pre) static_cast<T*>(p.e.pre)[t * p.e.ldp + c] = from_f32<T>(v);
        v = act_any(p.e.act, v);
        if (p.e.res) v += to_f32(static_cast<const T*>(p.e.res)[t * p.e.ldr + c]);
        static_cast<T*>(p.e.out)[t * p.e.ldo + c] = from_f32<T>(v);
      }
    }
    if (p.kw > 1) __syncthreads();
  }
}

template <typename T, int TT, bool VECTOR>
int run_few(FewArgs p, cudaStream_t st) {
  constexpr int R = TT <= 2 ? 2 : 1;
  // warps a row: enough rows for about 16 warps an SM, else share a row among more
  const int64_t want = 16 * int64_t(num_sms());
  p.kw = 1;
  while (p.kw < kWarpsG && (int64_t(p.N) + R - 1) / R * p.kw < want && p.K >= 256 * p.kw) p.kw *= 2;
  const int64_t groups = (int64_t(p.N) + int64_t(kWarpsG / p.kw) * R - 1) / (int64_t(kWarpsG / p.kw) * R);
  constexpr int copies = !VECTOR && TT == 1 ? 4 : TT;
  const size_t smem = size_t(copies) * few_pitch(p.K) * 4;
  auto kern = linear_few_kernel<T, TT, VECTOR, R>;
  if (smem > 40 * 1024) {
    static std::atomic<unsigned long long> seen{0};
    const int rc = allow_smem(reinterpret_cast<const void*>(kern), copies * few_pitch(kSliceK) * 4, seen);
    if (rc != MOE_OK) return rc;
  }
  // a whole number of row groups a CTA, about three CTAs an SM
  const int64_t most = 3 * int64_t(num_sms());
  const int64_t each = (groups + most - 1) / most;
  return launch_kernel(kern, dim3(unsigned((groups + each - 1) / each)), dim3(kThreadsG), smem, st, p);
}

int dispatch_f32(const FewArgs& p, bool vec, cudaStream_t st) {
  if (p.T == 1) return vec ? run_few<float, 1, true>(p, st) : run_few<float, 1, false>(p, st);
  if (p.T == 2) return vec ? run_few<float, 2, true>(p, st) : run_few<float, 2, false>(p, st);
  if (p.T <= 4) return vec ? run_few<float, 4, true>(p, st) : run_few<float, 4, false>(p, st);
  return vec ? run_few<float, 8, true>(p, st) : run_few<float, 8, false>(p, st);
}

}  // namespace

int launch_linear_few(int bf16, const void* x, int64_t ldx, const void* W, int64_t ldw, int T, int N, int K,
                      const LinearEpi& e, cudaStream_t st) {
  FewArgs p{x, W, ldx, ldw, T, N, K, 1, e};
  const int v = bf16 ? 8 : 4;
  const bool vec = reinterpret_cast<uintptr_t>(W) % 16 == 0 && ldw % v == 0 && K % v == 0;
  if (!bf16) return dispatch_f32(p, vec, st);
  if (T != 1) return MOE_ERR_UNSUPPORTED;
  return vec ? run_few<__nv_bfloat16, 1, true>(p, st) : run_few<__nv_bfloat16, 1, false>(p, st);
}

}  // namespace moe
