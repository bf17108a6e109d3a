// The tensor-core products (linear_bf16.cuh) of the cross entropy of a linear head.
#include "linear_bf16.cuh"

namespace moe {
namespace {

// out (fp32, or times the factor and rounded to bf16) = the sums of the splits, in their order, + acc_in. A thread
// takes 8 columns of a row.
__global__ void __launch_bounds__(256) product_join_kernel(const XentEpi x, int rows, int cols, void* out, int64_t ldo) {
  pdl_wait();
  pdl_trigger();
  const int64_t groups = x.ldacc / 8, n = rows * groups, all = int64_t(rows) * x.ldacc;
  const float f = x.acc_out ? 1.f : xent_factor(x);
  const bool vec = reinterpret_cast<uintptr_t>(out) % 16 == 0 && ldo % 8 == 0;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto add = [&](const float* p) {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
      v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    };
    if (x.acc_in) add(x.acc_in + i * 8);
#pragma unroll 4
    for (int s = 0; s < x.splits; ++s) add(x.sums + s * all + i * 8);
    if (x.acc_out) {
      float4* o = reinterpret_cast<float4*>(x.acc_out + i * 8);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
      continue;
    }
    const int64_t row = i / groups;
    const int c = int(i - row * groups) * 8;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + row * ldo + c;
    if (vec && c + 8 <= cols) {
      *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f),
                                                pack_bf16x2(v[4] * f, v[5] * f), pack_bf16x2(v[6] * f, v[7] * f));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < cols) o[q] = __float2bfloat16_rn(v[q] * f);
    }
  }
}

constexpr int kPairs = 76;  // SM pairs of a GB300
constexpr size_t kSumBytes = size_t(96) << 20;

}  // namespace

// An estimate in units of a pair's k-block (0.365 us for 256 x 256 x 64 at the sustained rate), for the whole reduction at
// once and for s parts: rounds of tiles over the pairs, 14 blocks of start and end a round, and for the parts
// their sums' way through memory (0.22 blocks a tile and part) and the joining launch (12 blocks). Undivided, outputs
// with fewer tiles than half of the pairs take 128 x 128 tiles on single CTAs, in up to 8 splits of their own:
// 0.28 us a k-block. dx of 1003 x 1411 over 20011: 107 us in tiles, 44 in 3 parts.
int product_sum_splits(int rows, int cols, int K) {
  if (rows <= 64 || cols < 128) return 1;
  const int64_t tiles = ((int64_t(rows) + 255) / 256) * ((int64_t(cols) + 255) / 256), nkb = (int64_t(K) + 63) / 64;
  const int64_t small = ((int64_t(rows) + 127) / 128) * ((int64_t(cols) + 127) / 128);
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  double best;
  if (2 * tiles >= kPairs) {
    best = double(up(tiles, kPairs)) * double(nkb + 14);
  } else {
    int64_t s = 1;
    while (s < 8 && small * s * 2 <= 2 * kPairs * 7 / 8 && nkb >= 8 * s) s *= 2;
    best = 0.77 * double(up(small * s, 2 * kPairs)) * double(up(nkb, s) + 20);
  }
  int pick = 1;
  for (int s = 2; s <= 64; ++s) {
    if (nkb < 8 * int64_t(s) || size_t(s) * rows * up8(cols) * 4 > kSumBytes) break;
    const double t = double(up(tiles * s, kPairs)) * double(up(nkb, s) + 14) + 12.0 + 0.22 * double(tiles * s);
    if (t < 0.97 * best) {
      best = t;
      pick = s;
    }
  }
  return pick;
}

int xent_stats_cols(int rows, int cols) { return takes_pairs(rows, cols, false) ? 256 : 128; }

int launch_xent_bf16(ProductMode mode, const LinearOperand& A, const LinearOperand& B, int rows, int cols, int K,
                     const LinearEpi& e, const XentEpi& x, unsigned* status, cudaStream_t st) {
  switch (mode) {
    case kXentStats: return run_product<kXentStats>(A, B, rows, cols, K, e, x, status, st);
    case kXentGrad: return run_product<kXentGrad>(A, B, rows, cols, K, e, x, status, st);
    case kProductSum: {
      const int rc = run_product<kProductSum>(A, B, rows, cols, K, e, x, status, st);
      if (rc != MOE_OK || x.splits == 1) return rc;
      const int64_t n = int64_t(rows) * (x.ldacc / 8);
      return launch_kernel(product_join_kernel, dim3(unsigned(std::min<int64_t>((n + 255) / 256, 8 * num_sms()))),
                           dim3(256), 0, st, x, rows, cols, e.out, e.ldo);
    }
    case kProduct: break;
  }
  return MOE_ERR_INVALID_ARG;
}

}  // namespace moe
