// The linear layer's products in fp32 on plain FMA (a tensor-core product of rounded inputs
// cannot meet an fp32 tolerance).
//
//   out(i, j) = act(sum_k A(i, k) B(j, k) + bias[j]) + residual(i, j)
//
// for the forward (A = x, B = W), dx (A = d, B = W^T) and dW (A = d^T, B = x^T): the operands
// come with two strides, one of them 1, and are transposed on their way into shared memory.
// A CTA of 256 threads computes a 128 x 128 tile, 8 x 8 outputs a thread, over 16-deep slices
// of K, the next slice's loads in registers while the present one is multiplied. When the
// tiles are fewer than the SMs the K range is split over grid.z; the partial tiles are then
// added in split order by a second kernel, which applies the epilogue.
#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace {

constexpr int kTile = 128, kDepth = 16, kThreadsF = 256;
constexpr int kPitch = kTile + 4;

struct Operand {
  const float* p;
  int64_t si, sk;  // strides of the row (i or j) and of k
  int rows;
  int vec;  // 16-byte loads along the unit stride are possible
};

// This thread's 8 values of the 128 x 16 slice: along k (unit sk) row tid / 2, k 8 (tid & 1)
// ..; along the rows (unit si) k tid / 16, rows 8 (tid & 15) ..
__device__ __forceinline__ void load_slice(const Operand& o, int r0, int64_t k0, int64_t k1, float (&v)[8]) {
  const int tid = threadIdx.x;
  if (o.sk == 1) {
    const int r = r0 + (tid >> 1);
    const int64_t k = k0 + 8 * (tid & 1);
    const float* p = o.p + r * o.si + k;
    if (r < o.rows && o.vec && k + 8 <= k1) {
      *reinterpret_cast<float4*>(v) = __ldg(reinterpret_cast<const float4*>(p));
      *reinterpret_cast<float4*>(v + 4) = __ldg(reinterpret_cast<const float4*>(p + 4));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = (r < o.rows && k + q < k1) ? __ldg(p + q) : 0.f;
    }
  } else {
    const int r = r0 + 8 * (tid & 15);
    const int64_t k = k0 + (tid >> 4);
    const float* p = o.p + r + k * o.sk;
    if (k < k1 && o.vec && r + 8 <= o.rows) {
      *reinterpret_cast<float4*>(v) = __ldg(reinterpret_cast<const float4*>(p));
      *reinterpret_cast<float4*>(v + 4) = __ldg(reinterpret_cast<const float4*>(p + 4));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = (k < k1 && r + q < o.rows) ? __ldg(p + q) : 0.f;
    }
  }
}
__device__ __forceinline__ void store_slice(const Operand& o, float* s, const float (&v)[8]) {
  const int tid = threadIdx.x;
  if (o.sk == 1) {
    const int r = tid >> 1, k = 8 * (tid & 1);
#pragma unroll
    for (int q = 0; q < 8; ++q) s[(k + q) * kPitch + r] = v[q];
  } else {
    float* d = s + (tid >> 4) * kPitch + 8 * (tid & 15);
    *reinterpret_cast<float4*>(d) = *reinterpret_cast<const float4*>(v);
    *reinterpret_cast<float4*>(d + 4) = *reinterpret_cast<const float4*>(v + 4);
  }
}

template <int ACT>
__device__ __forceinline__ void emit(const LinearEpi& e, int64_t i, int64_t j, float v) {
  if (e.bias) v += e.bias[j];
  if (e.pre) static_cast<float*>(e.pre)[i * e.ldp + j] = v;
  v = act_value<ACT>(v);
  if (e.res) v += static_cast<const float*>(e.res)[i * e.ldr + j];
  static_cast<float*>(e.out)[i * e.ldo + j] = v;
}

template <int ACT>
__global__ void __launch_bounds__(kThreadsF)
    linear_f32_kernel(Operand A, Operand B, int K, int kchunk, float* part, LinearEpi e) {
  __shared__ __align__(16) float sA[2][kDepth * kPitch], sB[2][kDepth * kPitch];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
  const int64_t k0 = int64_t(blockIdx.z) * kchunk, k1 = min(int64_t(K), k0 + kchunk);
  float acc[8][8];
#pragma unroll
  for (int a = 0; a < 8; ++a)
#pragma unroll
    for (int b = 0; b < 8; ++b) acc[a][b] = 0.f;
  float va[8], vb[8];
  load_slice(A, i0, k0, k1, va);
  load_slice(B, j0, k0, k1, vb);
  store_slice(A, sA[0], va);
  store_slice(B, sB[0], vb);
  __syncthreads();
  int buf = 0;
  for (int64_t k = k0; k < k1; k += kDepth) {
    const bool more = k + kDepth < k1;
    if (more) {
      load_slice(A, i0, k + kDepth, k1, va);
      load_slice(B, j0, k + kDepth, k1, vb);
    }
    const float* pa = sA[buf] + ty * 4;
    const float* pb = sB[buf] + tx * 4;
#pragma unroll
    for (int q = 0; q < kDepth; ++q) {
      float a[8], b[8];
      *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(pa + q * kPitch);
      *reinterpret_cast<float4*>(a + 4) = *reinterpret_cast<const float4*>(pa + q * kPitch + 64);
      *reinterpret_cast<float4*>(b) = *reinterpret_cast<const float4*>(pb + q * kPitch);
      *reinterpret_cast<float4*>(b + 4) = *reinterpret_cast<const float4*>(pb + q * kPitch + 64);
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[r][c] = fmaf(a[r], b[c], acc[r][c]);
    }
    if (more) {
      store_slice(A, sA[buf ^ 1], va);
      store_slice(B, sB[buf ^ 1], vb);
    }
    __syncthreads();
    buf ^= 1;
  }
  // thread (ty, tx): rows 4 ty .. + 3 and 64 + 4 ty .., columns likewise
  float* pt = part ? part + int64_t(blockIdx.z) * A.rows * B.rows : nullptr;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const int64_t i = i0 + (r >> 2) * 64 + ty * 4 + (r & 3);
    if (i >= A.rows) continue;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int64_t j = j0 + (c >> 2) * 64 + tx * 4 + (c & 3);
      if (j >= B.rows) continue;
      if (pt) pt[i * B.rows + j] = acc[r][c];
      else emit<ACT>(e, i, j, acc[r][c]);
    }
  }
}

template <int ACT>
__global__ void __launch_bounds__(256)
    linear_f32_join_kernel(const float* __restrict__ part, int splits, int rows, int cols, LinearEpi e) {
  pdl_wait();
  pdl_trigger();
  const int64_t n = int64_t(rows) * cols;
  for (int64_t x = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; x < n; x += int64_t(gridDim.x) * blockDim.x) {
    float v = 0.f;
    for (int s = 0; s < splits; ++s) v += part[s * n + x];
    emit<ACT>(e, x / cols, x % cols, v);
  }
}

Operand operand(const float* p, int64_t si, int64_t sk, int rows) {
  Operand o{p, si, sk, rows, 0};
  const int64_t ld = sk == 1 ? si : sk;
  o.vec = (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 4 == 0) ? 1 : 0;
  return o;
}

}  // namespace

int launch_linear_f32(const float* A, int64_t a_i, int64_t a_k, const float* B, int64_t b_j,
                      int64_t b_k, int rows, int cols, int K, const LinearEpi& e, float* part,
                      cudaStream_t st) {
  const Operand oa = operand(A, a_i, a_k, rows), ob = operand(B, b_j, b_k, cols);
  const int64_t ty = (rows + kTile - 1) / kTile, tx = (cols + kTile - 1) / kTile;
  if (ty > 65535) return MOE_ERR_UNSUPPORTED;
  // splits: about two tiles an SM, at least 64 deep each, within the scratch
  int splits = 1;
  if (tx * ty < num_sms()) {
    splits = int(std::min<int64_t>(std::min<int64_t>(2 * num_sms(), kPartTiles) / (tx * ty), (K + 63) / 64));
    if (splits < 1) splits = 1;
  }
  const int kchunk = int(((K + splits - 1) / splits + kDepth - 1) / kDepth * kDepth);
  splits = (K + kchunk - 1) / kchunk;
  return with_act(e.act, [&](auto tag) {
    constexpr int ACT = decltype(tag)::value;
    int rc = launch_kernel(linear_f32_kernel<ACT>, dim3(unsigned(tx), unsigned(ty), unsigned(splits)),
                           dim3(kThreadsF), 0, st, oa, ob, K, kchunk, splits > 1 ? part : nullptr, e);
    if (rc != MOE_OK || splits == 1) return rc;
    const int64_t n = int64_t(rows) * cols;
    const unsigned grid = unsigned(std::min<int64_t>((n + 255) / 256, 8 * num_sms()));
    return launch_kernel(linear_f32_join_kernel<ACT>, dim3(grid), dim3(256), 0, st,
                         static_cast<const float*>(part), splits, rows, cols, e);
  });
}

}  // namespace moe
