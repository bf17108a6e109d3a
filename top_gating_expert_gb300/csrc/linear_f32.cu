// The linear layer's products in fp32 on plain FMA (a tensor-core product of rounded inputs
// cannot meet an fp32 tolerance).
//
//   out(i, j) = act(sum_k A(i, k) B(j, k) + bias[j]) + residual(i, j)
//
// for the forward (A = x, B = W), dx (A = d, B = W^T) and dW (A = d^T, B = x^T): the operands
// come with two strides, one of them 1 (a template argument each: 3 % over reading them at run time),
// and are transposed on their way into shared memory, 64 bytes of a row by neighbouring lanes.
// A CTA of 256 threads computes a 128 x 128 tile, 8 x 8 outputs a thread as pairs of columns (two
// multiply-adds an instruction: with single ones the issue slots of shared-memory loads and
// multiply-adds together bound it), over 16-deep slices of K, the next slice's loads in registers while
// the present one is multiplied; two CTAs an SM. An output with a side of at most 64, 32 or 16 takes
// tiles of 64, 32 or 16 x 128 along it (linear_f32_narrow_kernel), rows and columns changing places where the
// columns are the short side: 16384 x 16 x 4096 forward 96 us (365 in whole tiles; 268 MB of x, 40 us),
// 16384 x 64 x 8192 420 (718), 16 x 4096 x 4096 25 us (61). When the
// tiles are fewer than half of what the SMs hold, the K range is split over grid.z; the partial tiles
// are then added in split order by a second kernel, which applies the epilogue. 2048^3: 349 us, 49
// TFLOP/s (the library's product 293): the multiply-adds' rate (213 us), 256 tiles on 304 places, and
// the waits on shared memory of four warps a scheduler bound it. (8 x 16 outputs a thread with half
// the threads: 388 us.)
#include <algorithm>
#include <type_traits>

#include "linear.cuh"

namespace moe {
namespace {

constexpr int kTile = 128, kDepth = 16, kThreadsF = 256;
// CTAs of ROWS x 128 tiles that an SM is to hold (their registers allow it)
// (16384 x 16 x 4096 with four, at 64 registers a thread, 106 us, with three 96; 2000 x 50 x 5000 with
// three 37.5, with two 33.4)
constexpr int ctas_per_sm(int rows) { return rows > 32 ? 2 : 3; }

constexpr int64_t kGridY = 65535;  // rows of tiles that one launch takes

struct Operand {
  const float* p;
  int64_t si, sk;  // strides of the row (i or j) and of k
  int rows;
  int vec;  // 16-byte loads along the unit stride are possible
};

// This thread's VALS = ROWS / 16 values of a ROWS x 16 slice: along k (unit sk) W consecutive k of a row
// (and of the row 64 on); along the rows (unit si) one k's consecutive rows.
template <int ROWS>
struct Slice {
  static constexpr int VALS = ROWS / 16, W = VALS < 4 ? VALS : 4, PER = 16 / W, PITCH = ROWS + 4;
};
template <int W>
__device__ __forceinline__ void load_whole(float* v, const float* p) {
  if constexpr (W == 4) *reinterpret_cast<float4*>(v) = __ldg(reinterpret_cast<const float4*>(p));
  else if constexpr (W == 2) *reinterpret_cast<float2*>(v) = __ldg(reinterpret_cast<const float2*>(p));
  else v[0] = __ldg(p);
}
template <int ROWS, bool ALONG_K>
__device__ __forceinline__ void load_slice(const Operand& o, int r0, int64_t k0, int64_t k1,
                                           float (&v)[ROWS / 16]) {
  using S = Slice<ROWS>;
  const int tid = threadIdx.x;
  if constexpr (ALONG_K) {
    const int64_t k = k0 + S::W * (tid % S::PER);
#pragma unroll
    for (int m = 0; m < S::VALS; m += S::W) {
      const int r = r0 + tid / S::PER + 16 * m;
      const float* p = o.p + r * o.si + k;
      if (r < o.rows && k + S::W <= k1 && o.vec) {
        load_whole<S::W>(v + m, p);
      } else {
#pragma unroll
        for (int q = 0; q < S::W; ++q) v[m + q] = r < o.rows && k + q < k1 ? __ldg(p + q) : 0.f;
      }
    }
  } else {
    const int r = r0 + S::VALS * (tid & 15);
    const int64_t k = k0 + (tid >> 4);
    const float* p = o.p + k * o.sk + r;
    if (k < k1 && r + S::VALS <= o.rows && o.vec) {
#pragma unroll
      for (int m = 0; m < S::VALS; m += S::W) load_whole<S::W>(v + m, p + m);
    } else {
#pragma unroll
      for (int q = 0; q < S::VALS; ++q) v[q] = k < k1 && r + q < o.rows ? __ldg(p + q) : 0.f;
    }
  }
}
template <int ROWS, bool ALONG_K>
__device__ __forceinline__ void store_slice(float* s, const float (&v)[ROWS / 16]) {
  using S = Slice<ROWS>;
  const int tid = threadIdx.x;
  if constexpr (ALONG_K) {
    float* d = s + S::W * (tid % S::PER) * S::PITCH + tid / S::PER;
#pragma unroll
    for (int m = 0; m < S::VALS; m += S::W)
#pragma unroll
      for (int q = 0; q < S::W; ++q) d[q * S::PITCH + 16 * m] = v[m + q];
  } else {
    float* d = s + (tid >> 4) * S::PITCH + S::VALS * (tid & 15);
    if constexpr (S::VALS >= 4) {
#pragma unroll
      for (int q = 0; q < S::VALS; q += 4) *reinterpret_cast<float4*>(d + q) = *reinterpret_cast<const float4*>(v + q);
    } else {
#pragma unroll
      for (int q = 0; q < S::VALS; ++q) d[q] = v[q];
    }
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

template <int ACT, bool AK, bool BK>  // AK, BK: the operand's unit stride is k's
__global__ void __launch_bounds__(kThreadsF, ctas_per_sm(kTile))
    linear_f32_kernel(Operand A, Operand B, int K, int kchunk, float* part, LinearEpi e) {
  constexpr int RT = 8, P = kTile + 4;  // rows a thread, pitch
  __shared__ __align__(16) float sA[2][kDepth * P], sB[2][kDepth * P];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile;
  const int64_t k0 = int64_t(blockIdx.z) * kchunk, k1 = min(int64_t(K), k0 + kchunk);
  f32x2 acc[RT][4];  // row r, column pairs
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = 0ull;
  float va[8], vb[8];
  load_slice<kTile, AK>(A, i0, k0, k1, va);
  load_slice<kTile, BK>(B, j0, k0, k1, vb);
  store_slice<kTile, AK>(sA[0], va);
  store_slice<kTile, BK>(sB[0], vb);
  __syncthreads();
  int buf = 0;
  for (int64_t k = k0; k < k1; k += kDepth) {
    const bool more = k + kDepth < k1;
    if (more) {
      load_slice<kTile, AK>(A, i0, k + kDepth, k1, va);
      load_slice<kTile, BK>(B, j0, k + kDepth, k1, vb);
    }
    const float* pa = sA[buf] + ty * 4;
    const float* pb = sB[buf] + tx * 4;
#pragma unroll
    for (int q = 0; q < kDepth; ++q) {
      float a[RT];
      *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(pa + q * P);
      *reinterpret_cast<float4*>(a + 4) = *reinterpret_cast<const float4*>(pa + q * P + 64);
      const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(pb + q * P);
      const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(pb + q * P + 64);
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
      store_slice<kTile, AK>(sA[buf ^ 1], va);
      store_slice<kTile, BK>(sB[buf ^ 1], vb);
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

// ROWS (16, 32 or 64) x 128 tiles, of the output's transpose with swap: 8 x 4 outputs a thread, so that
// 12 floats from shared memory feed 32 multiply-adds; the threads that this leaves over share a slice's
// k (64 / ROWS groups of them), and the groups' sums are added through shared memory in group order.
template <int ACT, int ROWS, bool AK, bool BK>
__global__ void __launch_bounds__(kThreadsF, ctas_per_sm(ROWS))
    linear_f32_narrow_kernel(Operand A, Operand B, int K, int kchunk, float* part, int swap, LinearEpi e) {
  constexpr int GROUPS = 64 / ROWS, DEPTH = kDepth / GROUPS, PA = ROWS + 4, PB = kTile + 4;
  constexpr int SLICE = kDepth * (PA + PB), SUMS = GROUPS * ROWS * PB;
  __shared__ __align__(16) float s_all[2 * SLICE > SUMS ? 2 * SLICE : SUMS];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, tx = tid & 31, ty = (tid >> 5) % (ROWS / 8), grp = tid / (4 * ROWS);
  const int i0 = blockIdx.y * ROWS, j0 = blockIdx.x * kTile;
  const int64_t k0 = int64_t(blockIdx.z) * kchunk, k1 = min(int64_t(K), k0 + kchunk);
  f32x2 acc[8][2];
#pragma unroll
  for (int a = 0; a < 8; ++a) acc[a][0] = acc[a][1] = 0ull;
  float va[ROWS / 16], vb[8];
  load_slice<ROWS, AK>(A, i0, k0, k1, va);
  load_slice<kTile, BK>(B, j0, k0, k1, vb);
  store_slice<ROWS, AK>(s_all, va);
  store_slice<kTile, BK>(s_all + kDepth * PA, vb);
  __syncthreads();
  int buf = 0;
  for (int64_t k = k0; k < k1; k += kDepth) {
    const bool more = k + kDepth < k1;
    if (more) {
      load_slice<ROWS, AK>(A, i0, k + kDepth, k1, va);
      load_slice<kTile, BK>(B, j0, k + kDepth, k1, vb);
    }
    const float* pa = s_all + buf * SLICE + grp * DEPTH * PA + ty * 8;
    const float* pb = s_all + buf * SLICE + kDepth * PA + grp * DEPTH * PB + tx * 4;
#pragma unroll
    for (int q = 0; q < DEPTH; ++q) {
      float a[8];
      *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(pa + q * PA);
      *reinterpret_cast<float4*>(a + 4) = *reinterpret_cast<const float4*>(pa + q * PA + 4);
      const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(pb + q * PB);
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const f32x2 aa = set2(a[r]);
        acc[r][0] = fma2(aa, b.x, acc[r][0]);
        acc[r][1] = fma2(aa, b.y, acc[r][1]);
      }
    }
    if (more) {
      store_slice<ROWS, AK>(s_all + (buf ^ 1) * SLICE, va);
      store_slice<kTile, BK>(s_all + (buf ^ 1) * SLICE + kDepth * PA, vb);
    }
    __syncthreads();
    buf ^= 1;
  }
  float* pt = part ? part + int64_t(blockIdx.z) * A.rows * B.rows : nullptr;
  if constexpr (GROUPS == 1) {
    auto leave = [&](auto swapped) {
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const int64_t i = i0 + ty * 8 + r;
        if (i >= A.rows) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int64_t j = j0 + tx * 4 + c;
          if (j >= B.rows) continue;
          const float2 f = unpack2(acc[r][c >> 1]);
          const float v = c & 1 ? f.y : f.x;
          if (pt) pt[i * B.rows + j] = v;
          else if (decltype(swapped)::value) emit<ACT>(e, j, i, v);
          else emit<ACT>(e, i, j, v);
        }
      }
    };
    return swap ? leave(std::bool_constant<true>{}) : leave(std::bool_constant<false>{});
  }
#pragma unroll
  for (int r = 0; r < 8; ++r)
    *reinterpret_cast<ulonglong2*>(s_all + (grp * ROWS + ty * 8 + r) * PB + tx * 4) =
        make_ulonglong2(acc[r][0], acc[r][1]);
  __syncthreads();
  const bool across = swap && !pt;  // consecutive threads along what is contiguous in the output
#pragma unroll
  for (int x = tid; x < ROWS * kTile; x += kThreadsF) {
    const int r = across ? x % ROWS : x / kTile, c = across ? x / ROWS : x % kTile;
    const int64_t i = i0 + r, j = j0 + c;
    if (i >= A.rows || j >= B.rows) continue;
    float v = s_all[r * PB + c];
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) v += s_all[(g * ROWS + r) * PB + c];
    if (pt) pt[i * B.rows + j] = v;
    else if (swap) emit<ACT>(e, j, i, v);
    else emit<ACT>(e, i, j, v);
  }
}

template <int ACT>
__global__ void __launch_bounds__(256)
    linear_f32_join_kernel(const float* __restrict__ part, int splits, int rows, int cols, int swap, LinearEpi e) {
  pdl_wait();
  pdl_trigger();
  const int64_t n = int64_t(rows) * cols;
  for (int64_t x = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; x < n; x += int64_t(gridDim.x) * blockDim.x) {
    float v = 0.f;
    for (int s = 0; s < splits; ++s) v += part[s * n + x];
    const int64_t i = x / cols, j = x - i * cols;
    emit<ACT>(e, swap ? j : i, swap ? i : j, v);
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
  // the shorter side of the output along the tiles' rows, in the smallest tile that holds it
  const int swap = cols < rows && cols <= 64;
  Operand oa = operand(A, a_i, a_k, rows), ob = operand(B, b_j, b_k, cols);
  if (swap) std::swap(oa, ob);
  const int tile_rows = oa.rows <= 16 ? 16 : (oa.rows <= 32 ? 32 : (oa.rows <= 64 ? 64 : kTile));
  const int64_t ty = (oa.rows + tile_rows - 1) / tile_rows, tx = (ob.rows + kTile - 1) / kTile;
  if (ty > kGridY) {  // (not swapped: a swapped side has 64 rows at most)
    const int most = int(kGridY) * kTile;
    for (int r = 0; r < rows; r += most) {
      LinearEpi part_e = e;
      part_e.out = static_cast<float*>(e.out) + r * e.ldo;
      if (e.pre) part_e.pre = static_cast<float*>(e.pre) + r * e.ldp;
      if (e.res) part_e.res = static_cast<const float*>(e.res) + r * e.ldr;
      const int rc = launch_linear_f32(A + r * a_i, a_i, a_k, B, b_j, b_k, std::min(most, rows - r), cols, K, part_e,
                                       part, st);
      if (rc != MOE_OK) return rc;
    }
    return MOE_OK;
  }
  // splits: about as many tiles as the SMs hold, at least 64 deep each, within the scratch
  int splits = 1;
  const int64_t room = ctas_per_sm(tile_rows) * num_sms();
  if (tx * ty <= room / 2) {
    const int64_t most = std::min<int64_t>(room, kPartTiles * (kTile / tile_rows));
    splits = int(std::min<int64_t>(most / (tx * ty), (K + 63) / 64));
    if (splits < 1) splits = 1;
  }
  const int kchunk = int(((K + splits - 1) / splits + kDepth - 1) / kDepth * kDepth);
  splits = (K + kchunk - 1) / kchunk;
  int rc;
  auto go = [&](auto act, auto ak, auto bk) {
    constexpr int ACT = decltype(act)::value;
    constexpr bool AK = decltype(ak)::value, BK = decltype(bk)::value;
    const dim3 grid = dim3(unsigned(tx), unsigned(ty), unsigned(splits));
    float* const to = splits > 1 ? part : nullptr;
    auto narrow = [&](auto kern) {
      return launch_kernel(kern, grid, dim3(kThreadsF), 0, st, oa, ob, K, kchunk, to, swap, e);
    };
    if (tile_rows == 16) return narrow(linear_f32_narrow_kernel<ACT, 16, AK, BK>);
    if (tile_rows == 32) return narrow(linear_f32_narrow_kernel<ACT, 32, AK, BK>);
    if (tile_rows == 64) return narrow(linear_f32_narrow_kernel<ACT, 64, AK, BK>);
    return launch_kernel(linear_f32_kernel<ACT, AK, BK>, grid, dim3(kThreadsF), 0, st, oa, ob, K, kchunk, to, e);
  };
  const bool ak = oa.sk == 1, bk = ob.sk == 1;
  constexpr std::bool_constant<true> yes{};
  constexpr std::bool_constant<false> no{};
  constexpr std::integral_constant<int, MOE_LIN_NONE> none{};  // the backward's products: no activation
  if (ak && bk) rc = with_act(e.act, [&](auto tag) { return go(tag, yes, yes); });
  else if (ak) rc = go(none, yes, no);
  else if (bk) rc = go(none, no, yes);
  else rc = go(none, no, no);
  if (rc != MOE_OK || splits == 1) return rc;
  const int64_t n = int64_t(rows) * cols;
  const unsigned grid = unsigned(std::min<int64_t>((n + 255) / 256, 8 * num_sms()));
  return with_act(e.act, [&](auto tag) {
    return launch_kernel(linear_f32_join_kernel<decltype(tag)::value>, dim3(grid), dim3(256), 0, st,
                         static_cast<const float*>(part), splits, oa.rows, ob.rows, swap, e);
  });
}

}  // namespace moe
