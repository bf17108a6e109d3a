// The linear layer's products in fp32 on plain FMA (a tensor-core product of rounded inputs
// cannot meet an fp32 tolerance).
//
//   out(i, j) = act(sum_k A(i, k) B(j, k) + bias[j]) + residual(i, j)
//
// for the forward (A = x, B = W), dx (A = d, B = W^T) and dW (A = d^T, B = x^T): the operands
// come with two strides, one of them 1, and are transposed on their way into shared memory.
// A CTA of 256 threads computes a 128 x 128 tile (64 x 128 for up to 64 rows), 8 x 8 outputs a
// thread as pairs of columns (two multiply-adds an instruction: with single ones the issue slots
// of shared-memory loads and multiply-adds together bound it), over 16-deep slices of K, the
// next slice's loads in registers while the present one is multiplied; two CTAs an SM. When the
// tiles are fewer than the SMs the K range is split over grid.z; the partial tiles are then
// added in split order by a second kernel, which applies the epilogue. 2048^3: 372 us, 46 TFLOP/s
// (the library's product 293): shared memory's rate and the 1.7 waves of 256 tiles bound it.
#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace {

constexpr int kTile = 128, kDepth = 16, kThreadsF = 256;

struct Operand {
  const float* p;
  int64_t si, sk;  // strides of the row (i or j) and of k
  int rows;
  int vec;  // 16-byte loads along the unit stride are possible
};

// This thread's VALS = ROWS / 16 values of a ROWS x 16 slice: along k (unit sk) a row's consecutive
// k; along the rows (unit si) one k's consecutive rows.
template <int ROWS>
__device__ __forceinline__ void load_slice(const Operand& o, int r0, int64_t k0, int64_t k1,
                                           float (&v)[ROWS / 16]) {
  constexpr int VALS = ROWS / 16, PER = 16 / VALS;  // threads along k of a row
  const int tid = threadIdx.x;
  const bool along_k = o.sk == 1;
  const int r = r0 + (along_k ? tid / PER : VALS * (tid & 15));
  const int64_t k = k0 + (along_k ? VALS * (tid % PER) : (tid >> 4));
  const float* p = o.p + r * o.si + k * o.sk;
  const bool whole = along_k ? (r < o.rows && k + VALS <= k1) : (k < k1 && r + VALS <= o.rows);
  if (whole && o.vec) {
#pragma unroll
    for (int q = 0; q < VALS; q += 4) *reinterpret_cast<float4*>(v + q) = __ldg(reinterpret_cast<const float4*>(p + q));
  } else {
#pragma unroll
    for (int q = 0; q < VALS; ++q)
      v[q] = (along_k ? (r < o.rows && k + q < k1) : (k < k1 && r + q < o.rows)) ? __ldg(p + q) : 0.f;
  }
}
template <int ROWS>
__device__ __forceinline__ void store_slice(const Operand& o, float* s, const float (&v)[ROWS / 16]) {
  constexpr int VALS = ROWS / 16, PER = 16 / VALS, PITCH = ROWS + 4;
  const int tid = threadIdx.x;
  if (o.sk == 1) {
    const int r = tid / PER, k = VALS * (tid % PER);
#pragma unroll
    for (int q = 0; q < VALS; ++q) s[(k + q) * PITCH + r] = v[q];
  } else {
    float* d = s + (tid >> 4) * PITCH + VALS * (tid & 15);
#pragma unroll
    for (int q = 0; q < VALS; q += 4) *reinterpret_cast<float4*>(d + q) = *reinterpret_cast<const float4*>(v + q);
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

template <int ACT, int ROWS>
__global__ void __launch_bounds__(kThreadsF, 2)
    linear_f32_kernel(Operand A, Operand B, int K, int kchunk, float* part, LinearEpi e) {
  constexpr int RT = ROWS / 16, PA = ROWS + 4, PB = kTile + 4;  // rows a thread, pitches
  __shared__ __align__(16) float sA[2][kDepth * PA], sB[2][kDepth * PB];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int i0 = blockIdx.y * ROWS, j0 = blockIdx.x * kTile;
  const int64_t k0 = int64_t(blockIdx.z) * kchunk, k1 = min(int64_t(K), k0 + kchunk);
  f32x2 acc[RT][4];  // row r, column pairs
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = 0ull;
  float va[RT], vb[8];
  load_slice<ROWS>(A, i0, k0, k1, va);
  load_slice<kTile>(B, j0, k0, k1, vb);
  store_slice<ROWS>(A, sA[0], va);
  store_slice<kTile>(B, sB[0], vb);
  __syncthreads();
  int buf = 0;
  for (int64_t k = k0; k < k1; k += kDepth) {
    const bool more = k + kDepth < k1;
    if (more) {
      load_slice<ROWS>(A, i0, k + kDepth, k1, va);
      load_slice<kTile>(B, j0, k + kDepth, k1, vb);
    }
    const float* pa = sA[buf] + ty * 4;
    const float* pb = sB[buf] + tx * 4;
#pragma unroll
    for (int q = 0; q < kDepth; ++q) {
      float a[RT];
#pragma unroll
      for (int h = 0; h < RT / 4; ++h)
        *reinterpret_cast<float4*>(a + 4 * h) = *reinterpret_cast<const float4*>(pa + q * PA + 64 * h);
      const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(pb + q * PB);
      const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(pb + q * PB + 64);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const f32x2 aa = set2(a[r]);
        acc[r][0] = fma2(aa, b0.x, acc[r][0]);
        acc[r][1] = fma2(aa, b0.y, acc[r][1]);
        acc[r][2] = fma2(aa, b1.x, acc[r][2]);
        acc[r][3] = fma2(aa, b1.y, acc[r][3]);
      }
    }
    if (more) {
      store_slice<ROWS>(A, sA[buf ^ 1], va);
      store_slice<kTile>(B, sB[buf ^ 1], vb);
    }
    __syncthreads();
    buf ^= 1;
  }
  // thread (ty, tx): rows 4 ty .. + 3 (and 64 + 4 ty ..), columns 4 tx .. and 64 + 4 tx ..
  float* pt = part ? part + int64_t(blockIdx.z) * A.rows * B.rows : nullptr;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int64_t i = i0 + (r >> 2) * 64 + ty * 4 + (r & 3);
    if (i >= A.rows) continue;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int64_t j = j0 + (c >> 2) * 64 + tx * 4 + (c & 3);
      if (j >= B.rows) continue;
      const float2 f = unpack2(acc[r][c >> 1]);
      const float v = c & 1 ? f.y : f.x;
      if (pt) pt[i * B.rows + j] = v;
      else emit<ACT>(e, i, j, v);
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
  const int tile_rows = rows <= 64 ? 64 : kTile;
  const int64_t ty = (rows + tile_rows - 1) / tile_rows, tx = (cols + kTile - 1) / kTile;
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
    auto kern = tile_rows == 64 ? linear_f32_kernel<ACT, 64> : linear_f32_kernel<ACT, kTile>;
    int rc = launch_kernel(kern, dim3(unsigned(tx), unsigned(ty), unsigned(splits)),
                           dim3(kThreadsF), 0, st, oa, ob, K, kchunk, splits > 1 ? part : nullptr, e);
    if (rc != MOE_OK || splits == 1) return rc;
    const int64_t n = int64_t(rows) * cols;
    const unsigned grid = unsigned(std::min<int64_t>((n + 255) / 256, 8 * num_sms()));
    return launch_kernel(linear_f32_join_kernel<ACT>, dim3(grid), dim3(256), 0, st,
                         static_cast<const float*>(part), splits, rows, cols, e);
  });
}

}  // namespace moe
