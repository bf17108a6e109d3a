// The linear layer's products in bf16 on the 5th-generation tensor cores (tcgen05 + TMEM,
// operands by TMA), fp32 accumulation, the epilogue applied to the fp32 sums:
//
//   out(i, j) = act(sum_k A(i, k) B(j, k) + bias[j]) + residual(i, j)
//
// for the forward (A = x, B = W), dx (A = d, B = W^T) and dW (A = d^T, B = x^T). Each operand
// is K-major (its rows contiguous along k) or MN-major (contiguous along i or j): the MMA
// reads either from the 128-byte-swizzled boxes that TMA writes, so nothing is transposed in
// memory. Rows, columns and k past the ends read as zeros (TMA's fill), so every size runs on
// the same path.
//
// linear_tile_kernel: one CTA per 128 x BN tile of D and per split of K.
//   warp 0      TMA producer (a ring of `stages` stages of 64-wide k-blocks)
//   warp 1      TMEM owner and MMA issuer
//   warps 2..5  move the finished accumulator into shared memory (over the drained ring)
//   all warps   epilogue: contiguous runs of an output row, 4 columns a thread
// With few rows (a serving step) the roles are exchanged (TRANS): the 128-row side is W and
// the narrow side the tokens, so the MMA's M is full and the kernel streams W. When the tiles are fewer than the SMs, K is split over the CTAs of a cluster;
// each then sums its share of the tile over the cluster's shared memories in split order, so
// the result does not depend on timing and no scratch in memory is needed.
// 777 x 1408 x 2048 (77 tiles, 32 k-blocks): 16 us, a k-block 0.28 us where the MMAs would take
// 0.16: bound by the operands' way from L2 (32 KB a k-block for 128 x 128 outputs). 64 x 14336 x
// 4096: 27 us, W at 4.3 TB/s on 112 of the 152 SMs.
//
// Every mbarrier wait is bounded, as in the grouped GEMM: a role that gives up sets the status word
// and the CTA's abort flag, the loads and MMAs in flight are drained, TMEM is freed.
#include <algorithm>
#include <type_traits>

#include "linear.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

using namespace sm100;

constexpr int BM = 128;
constexpr int BK = 64;  // bf16 elements of a 128-byte swizzled row
constexpr int kMaxStages = 8;

struct TileArgs {
  int rows, cols, nkb, splits, stages;
  int a_mn, b_mn;
  int vec;  // 8-byte accesses to bias, residual, pre and out rows
  LinearEpi e;
  unsigned* status;
};

__device__ __forceinline__ float ld_cluster_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Epilogue: a warp takes whole rows of the tile, a lane 4 consecutive columns (VEC: 8-byte
// accesses, when every row of every operand allows them) or every 32nd column. The residual's
// loads of several rows are issued before the first is used.
__device__ __forceinline__ float2 bf16x2_floats(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// Column of this lane's q-th value.
template <bool VEC>
__device__ __forceinline__ int lane_col(int lane, int q) {
  return VEC ? (q >> 2) * 128 + lane * 4 + (q & 3) : lane + 32 * q;
}

// Stores the valid ones of a row's values, 4 at a time when VEC.
template <int NC, bool VEC>
__device__ __forceinline__ void store_row(void* base, int64_t at, const float (&v)[NC], int lane, int nc) {
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(base) + at;
  if constexpr (VEC) {
#pragma unroll
    for (int q = 0; q < NC; q += 4)
      if (lane_col<true>(lane, q) < nc)  // 4 divides nc
        *reinterpret_cast<uint2*>(o + lane_col<true>(lane, q)) =
            make_uint2(pack_bf16x2(v[q], v[q + 1]), pack_bf16x2(v[q + 2], v[q + 3]));
  } else {
#pragma unroll
    for (int q = 0; q < NC; ++q)
      if (lane + 32 * q < nc) o[lane + 32 * q] = __float2bfloat16_rn(v[q]);
  }
}

// The epilogue of output rows r, r + step, .. (those below r_end, at most ROWS of them), columns
// c0 .. c0 + nc - 1; get(row, column of the tile) reads the summed accumulator.
template <int NC, int ROWS, bool VEC, typename Get>
__device__ __forceinline__ void emit_rows(const LinearEpi& e, int r, int step, int r_end, int64_t row0, int64_t c0,
                                          int nc, int lane, const float (&bias)[NC], Get&& get) {
  float v[ROWS][NC];
  uint2 rv[ROWS][VEC ? NC / 4 : 1];
  __nv_bfloat16 rs[ROWS][VEC ? 1 : NC];
  if (e.res) {
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      if (r + k * step >= r_end) break;
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(e.res) + (row0 + r + k * step) * e.ldr + c0;
      if constexpr (VEC) {
#pragma unroll
        for (int q = 0; q < NC; q += 4)
          if (lane_col<true>(lane, q) < nc) rv[k][q / 4] = *reinterpret_cast<const uint2*>(p + lane_col<true>(lane, q));
      } else {
#pragma unroll
        for (int q = 0; q < NC; ++q)
          if (lane + 32 * q < nc) rs[k][q] = p[lane + 32 * q];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    if (r + k * step >= r_end) break;
    get(r + k * step, v[k]);
#pragma unroll
    for (int q = 0; q < NC; ++q) v[k][q] += bias[q];
    const int64_t row = row0 + r + k * step;
    if (e.pre) store_row<NC, VEC>(e.pre, row * e.ldp + c0, v[k], lane, nc);
    act_fast_all(e.act, v[k]);
    if (e.res) {
#pragma unroll
      for (int q = 0; q < NC; ++q) {
        if (lane_col<VEC>(lane, q) >= nc) continue;
        if constexpr (VEC) {
          const float2 f = bf16x2_floats((q & 2) ? rv[k][q / 4].y : rv[k][q / 4].x);
          v[k][q] += (q & 1) ? f.y : f.x;
        } else {
          v[k][q] += __bfloat162float(rs[k][q]);
        }
      }
    }
    store_row<NC, VEC>(e.out, row * e.ldo + c0, v[k], lane, nc);
  }
}

template <int BN, bool TRANS>
struct TileCfg {
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_BYTES = BN * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int PITCH = (TRANS ? BM : BN) + 4;  // floats of a staged output row
  static constexpr int DUMP = (TRANS ? BN : BM) * PITCH * 4;
  static constexpr int TMEM_COLS = BN < 32 ? 32 : BN;
  // six more warps for the epilogue of 128 rows (a tile's epilogue is bound by latency)
  static constexpr int THREADS = TRANS ? 192 : 384;
};

template <int BN, bool TRANS>
__global__ void __launch_bounds__(TileCfg<BN, TRANS>::THREADS, TRANS ? 3 : 1)
    linear_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const TileArgs p) {
  using C = TileCfg<BN, TRANS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * kMaxStages + 1];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int NS = p.stages;
  uint8_t* sA = smem;
  uint8_t* sB = smem + NS * C::A_BYTES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages;
  const uint32_t done_bar = empty0 + 8 * kMaxStages;
  const int i0 = blockIdx.x * BM, j0 = blockIdx.y * BN;
  const int split = blockIdx.z;  // the CTA's rank in its cluster when splits > 1

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    mbar_init(done_bar, 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
  }
  if (warp == 1) tmem_alloc(smem_u32(&s_tmem), C::TMEM_COLS);
  // this split's k-blocks
  const int kb0 = int(int64_t(p.nkb) * split / p.splits);
  const int kb1 = int(int64_t(p.nkb) * (split + 1) / p.splits);
  if (TRANS && warp == 2 && lane == 0)  // few rows: the weights into L2 while the previous kernel ends
    for (int kb = kb0; kb < min(kb1, kb0 + NS); ++kb) {
      if (p.a_mn) {
        tma_prefetch_2d(&tmA, i0, kb * BK);
        if (i0 + 64 < p.rows) tma_prefetch_2d(&tmA, i0 + 64, kb * BK);
      } else {
        tma_prefetch_2d(&tmA, kb * BK, i0);
      }
    }
  pdl_wait();
  pdl_trigger();
  const uint64_t wlimit = wait_limit_ns(p.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  bool any = false;  // warp 0: loads issued; warp 1: MMAs issued
  int stage = 0;
  uint32_t phase = 0;
  uint32_t issued = 0, issued_par = 0;
  if (warp == 0) {
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = __all_sync(0xffffffffu, wait_bounded(empty0 + 8 * stage, phase ^ 1u, &s_abort, p.status, wlimit));
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = full0 + 8 * stage;
        const uint32_t dA = smem_u32(sA + stage * C::A_BYTES), dB = smem_u32(sB + stage * C::B_BYTES);
        mbar_expect_tx(fb, C::STAGE);
        if (p.a_mn) {
          tma_load_2d(dA, &tmA, i0, kb * BK, fb);
          tma_load_2d(dA + 8192, &tmA, i0 + 64, kb * BK, fb);
        } else {
          tma_load_2d(dA, &tmA, kb * BK, i0, fb);
        }
        if constexpr (BN >= 64) {
          if (p.b_mn) {
#pragma unroll
            for (int b = 0; b < BN / 64; ++b) tma_load_2d(dB + b * 8192, &tmB, j0 + 64 * b, kb * BK, fb);
          } else {
            tma_load_2d(dB, &tmB, kb * BK, j0, fb);
          }
        } else {
          tma_load_2d(dB, &tmB, kb * BK, j0, fb);
        }
      }
      __syncwarp();
      issued |= 1u << stage;
      issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
      if (++stage == NS) {
        stage = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16(BM, BN) | (p.a_mn ? 1u << 15 : 0u) | (p.b_mn ? 1u << 16 : 0u);
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      ok = __all_sync(0xffffffffu, wait_bounded(full0 + 8 * stage, phase, &s_abort, p.status, wlimit));
      if (!ok) break;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t a0 = smem_u32(sA + stage * C::A_BYTES), b0 = smem_u32(sB + stage * C::B_BYTES);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk) {
          const uint64_t ad = p.a_mn ? mn_sw128_desc(a0 + kk * 2048) : sw128_desc(a0 + kk * 32);
          const uint64_t bd = p.b_mn ? mn_sw128_desc(b0 + kk * 2048) : sw128_desc(b0 + kk * 32);
          mma_bf16(tmem, ad, bd, idesc, (kb != kb0 || kk != 0) ? 1u : 0u);
        }
        mma_commit(empty0 + 8 * stage);
      }
      __syncwarp();
      any = true;
      if (++stage == NS) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if (lane == 0 && any) mma_commit(done_bar);  // on a failure too: what was issued finishes
    __syncwarp();
  } else if (warp < 6) {
    const bool ok = __all_sync(0xffffffffu, wait_bounded(done_bar, 0u, &s_abort, p.status, wlimit));
    tc_fence_after();
    if (ok) {
      const int q = warp & 3, row = 32 * q + lane;  // this lane's accumulator row
      float* dump = reinterpret_cast<float*>(smem);
      const uint32_t tbase = tmem + (uint32_t(q * 32) << 16);
#pragma unroll 1
      for (int c0 = 0; c0 < BN; c0 += 16) {
        uint32_t v[16];
        tmem_ld16(tbase + c0, v);
        tmem_ld_wait();
        if constexpr (TRANS) {
#pragma unroll
          for (int x = 0; x < 16; ++x) dump[(c0 + x) * C::PITCH + row] = __uint_as_float(v[x]);
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4*>(dump + row * C::PITCH + c0 + 4 * x) =
                make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (s_abort) {
    // loads issued land and MMAs issued finish before shared and tensor memory go away
    if (warp == 0 && lane == 0)
      for (int s = 0; s < NS; ++s)
        if ((issued >> s) & 1u) wait_drain(full0 + 8 * s, (issued_par >> s) & 1u);
    if (warp == 1 && any) wait_drain(done_bar, 0u);
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (p.splits > 1) cluster_sync_all();  // every split's tile is in its shared memory

  // epilogue: this CTA's share of the output rows of the tile
  constexpr int OR = TRANS ? BN : BM, OC = 128, NC = OC / 32;
  const int or0 = OR * split / p.splits;
  const int r0 = TRANS ? j0 : i0, c0 = TRANS ? i0 : j0;
  const int nr = TRANS ? p.cols : p.rows, nc = min(OC, (TRANS ? p.rows : p.cols) - c0);
  const int or1 = min(OR * (split + 1) / p.splits, nr - r0);
  const uint32_t base = smem_u32(smem);
  auto run = [&](auto vec) {
    constexpr bool VEC = decltype(vec)::value;
    float bias[NC];
#pragma unroll
    for (int q = 0; q < NC; ++q)
      bias[q] = p.e.bias && lane_col<VEC>(lane, q) < nc ? __ldg(p.e.bias + c0 + lane_col<VEC>(lane, q)) : 0.f;
    auto get = [&](int r, float (&v)[NC]) {
#pragma unroll
      for (int q = 0; q < NC; q += VEC ? 4 : 1) {
        const uint32_t off = uint32_t(r * C::PITCH + lane_col<VEC>(lane, q)) * 4;
        if (p.splits > 1) {
#pragma unroll
          for (int x = 0; x < (VEC ? 4 : 1); ++x) v[q + x] = 0.f;
          for (int s = 0; s < p.splits; ++s) {
            const uint32_t at = cluster_addr(base + off, uint32_t(s));
            if constexpr (VEC) {
              const float4 f = ld_cluster_f4(at);
              v[q] += f.x; v[q + 1] += f.y; v[q + 2] += f.z; v[q + 3] += f.w;
            } else {
              v[q] += ld_cluster_f(at);
            }
          }
        } else if constexpr (VEC) {
          const float4 f = *reinterpret_cast<const float4*>(smem + off);
          v[q] = f.x; v[q + 1] = f.y; v[q + 2] = f.z; v[q + 3] = f.w;
        } else {
          v[q] = *reinterpret_cast<const float*>(smem + off);
        }
      }
    };
    constexpr int ROWS = 4, W = C::THREADS / 32;
    for (int r = or0 + warp; r < or1; r += ROWS * W)
      emit_rows<NC, ROWS, VEC>(p.e, r, W, or1, r0, c0, nc, lane, bias, get);
  };
  if (p.vec) run(std::true_type{});
  else run(std::false_type{});
  __syncwarp();
  if (p.splits > 1) cluster_sync_all();  // no CTA leaves while another reads its tile
}

int map_operand(CUtensorMap* m, const LinearOperand& o, int rows, int K, int box) {
  return o.mn ? make_tma_map_strided(m, o.p, K, rows, o.ld, 64)
              : make_tma_map_strided(m, o.p, rows, K, o.ld, box);
}

template <int BN, bool TRANS>
int run_tile(const LinearOperand& A, const LinearOperand& B, int rows, int cols, int K, int splits,
             const LinearEpi& e, unsigned* status, cudaStream_t st) {
  using C = TileCfg<BN, TRANS>;
  if (B.mn && BN < 64) return MOE_ERR_UNSUPPORTED;
  CUtensorMap ta, tb;
  int rc;
  if ((rc = map_operand(&ta, A, rows, K, BM)) != MOE_OK) return rc;
  if ((rc = map_operand(&tb, B, cols, K, BN)) != MOE_OK) return rc;
  TileArgs p;
  p.rows = rows; p.cols = cols;
  p.nkb = (K + BK - 1) / BK;
  p.splits = splits;
  p.a_mn = A.mn; p.b_mn = B.mn;
  p.e = e;
  p.status = status;
  // CTAs an SM: as many as the grid brings, while each still has three stages and room for the
  // staged tile (the stages in flight of all of them are what hides the memory's latency)
  const int64_t ctas = int64_t((rows + BM - 1) / BM) * ((cols + BN - 1) / BN) * splits;
  int per_sm = int(std::min<int64_t>(3, (ctas + num_sms() - 1) / num_sms()));
  auto stages_at = [](int n) { return std::min(kMaxStages, (233472 / n - 1024 - 1024 - 512) / C::STAGE); };
  while (per_sm > 1 && (stages_at(per_sm) < 3 || stages_at(per_sm) * C::STAGE < C::DUMP)) --per_sm;
  p.stages = stages_at(per_sm);
  const int smem = 1024 + p.stages * C::STAGE;
  if (p.stages * C::STAGE < C::DUMP) return MOE_ERR_UNSUPPORTED;
  const int64_t oc = TRANS ? rows : cols;
  auto vec8 = [](const void* q, int64_t ld) { return !q || (reinterpret_cast<uintptr_t>(q) % 8 == 0 && ld % 4 == 0); };
  p.vec = oc % 4 == 0 && vec8(e.out, e.ldo) && vec8(e.pre, e.ldp) && vec8(e.res, e.ldr);
  auto kern = linear_tile_kernel<BN, TRANS>;
  static std::atomic<unsigned long long> seen{0};
  if ((rc = allow_smem(reinterpret_cast<const void*>(kern), 1024 + stages_at(1) * C::STAGE, seen)) != MOE_OK)
    return rc;
  cudaLaunchConfig_t lc = {};
  const int64_t tj = (int64_t(cols) + BN - 1) / BN;
  if (tj > 65535) return MOE_ERR_UNSUPPORTED;
  lc.gridDim = dim3(unsigned((rows + BM - 1) / BM), unsigned(tj), unsigned(splits));
  lc.blockDim = dim3(C::THREADS);
  lc.dynamicSmemBytes = smem;
  lc.stream = st;
  cudaLaunchAttribute attr[2];
  lc.attrs = attr;
  lc.numAttrs = 0;
  if (splits > 1) {
    attr[lc.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[lc.numAttrs].val.clusterDim.x = 1;
    attr[lc.numAttrs].val.clusterDim.y = 1;
    attr[lc.numAttrs].val.clusterDim.z = unsigned(splits);
    ++lc.numAttrs;
  }
  if (pdl_enabled()) {
    attr[lc.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[lc.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++lc.numAttrs;
  }
  MOE_CUDA_CHECK(cudaLaunchKernelEx(&lc, kern, ta, tb, p));
  return MOE_OK;
}

// ------------------------------------------------------------------ large products
// linear_pair_kernel: persistent, one cluster of two CTAs per pair of SMs, each walking output
// tiles of 256 x BN (cta_group::2 MMAs: every CTA stages its 128 rows of A and its half of B's
// BN rows, so an SM pulls 32 KB per 64-wide k-block for 128 x 256 outputs).
//   warp 0      TMA producer; both CTAs' loads complete on the even CTA's `full` barrier
//   warp 1      TMEM owner; the even CTA's issues the MMAs into one of two accumulators
//   warps 2..9  epilogue, two warps per 32 TMEM lanes, each half of the columns: 32 columns at
//               a time from TMEM through bias, activation and residual into a swizzled 32 x 32
//               box in shared memory and out by a TMA store (two boxes a warp in turn). The
//               next tile's MMAs run meanwhile.
// Tiles are walked in bands of kBand tile rows, column by column, so that the tiles in
// flight share their operands through L2 (bands of 8 the same, 4 and 32 slower by 3 and 11 %).
//
// Measured: 8192 x 14336 x 4096 without epilogue 550 us (1.75 PFLOP/s, the library's product 542; 1.01
// of the sustained rate); bias adds 9 us, gelu 19 and the stored pre 21 (235 MB more), 607 us
// in all (0.92 of the sustained rate, the tensor pipe 84 % active in a capture). The backward's
// products at 16384 x 4096 x 1024 take 87 us each: 256 and 64 tiles fill 76 pairs to 84 %.
constexpr int kBand = 16;
constexpr int kPairThreads = 64 + 32 * 8;

struct PairArgs {
  int rows, cols, nkb, tiles_m, tiles_n;
  int a_mn, b_mn, res_vec, bias_vec;
  int res_tma;  // the residual comes by TMA (16-byte rows; not beside a stored pre, which takes the boxes)
  int stream;  // outputs too large to be found in L2 again: stores marked evict-first
  LinearEpi e;
  unsigned* status;
};

template <int BN>
struct PairCfg {
  static constexpr int A_BYTES = BM * BK * 2;
  static constexpr int B_BYTES = BN / 2 * BK * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int BOXES = 8 * 2 * 2048;  // 8 warps x 2 boxes of 32 x 32 bf16
  static constexpr int BARS = 512;
  static constexpr int STAGES = (232448 - 1024 - BOXES - BARS) / STAGE > 8 ? 8 : (232448 - 1024 - BOXES - BARS) / STAGE;
  static constexpr int SMEM = 1024 + STAGES * STAGE + BOXES + BARS;
  static constexpr int TMEM_COLS = 2 * BN;
};

template <int BN>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmP,
                       const __grid_constant__ CUtensorMap tmR, const PairArgs p) {
  using C = PairCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::STAGES * C::A_BYTES;
  uint8_t* sBox = sB + C::STAGES * C::B_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sBox + C::BOXES);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * C::STAGES + 5 + 16);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  volatile uint32_t* s_peer = s_tmem + 2;  // written by the other CTA at its end: k-blocks loaded, gave up
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::STAGES;
  const uint32_t tfull0 = empty0 + 8 * C::STAGES, tempty0 = tfull0 + 16, drain_bar = tempty0 + 16;
  const uint32_t res0 = drain_bar + 8;  // [8 warps][2 boxes]: a residual box has landed
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int unit = int(blockIdx.x >> 1), units = int(gridDim.x >> 1);
  const int total = p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, 8 * 2);
    }
    mbar_init(drain_bar, 1);
    for (int b = 0; b < 16; ++b) mbar_init(res0 + 8 * b, 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
    tma_prefetch_map(&tmY);
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(s_tmem), C::TMEM_COLS);
  pdl_wait();
  pdl_trigger();
  const uint64_t wlimit = wait_limit_ns(p.status);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers initialised in both CTAs
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  auto decode = [&](int t, int& m, int& n) {
    const int per = kBand * p.tiles_n, band = t / per, r = t - band * per;
    const int gm = min(kBand, p.tiles_m - band * kBand);
    n = r / gm;
    m = band * kBand + r - n * gm;
  };

  uint32_t issued = 0;  // warp 0: k-blocks loaded
  bool mma_any = false, mma_drained = false;
  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = unit; t < total && ok; t += units) {
      int m, n;
      decode(t, m, n);
      const int arow = m * 2 * BM + int(rank) * BM, brow = n * BN + int(rank) * (BN / 2);
      for (int kb = 0; kb < p.nkb; ++kb) {
        ok = __all_sync(0xffffffffu, wait_bounded(empty0 + 8 * stage, phase ^ 1u, s_abort, p.status, wlimit));
        if (!ok) break;
        if (lane == 0) {
          const uint32_t fb = full0 + 8 * stage, bar = cluster_addr(fb, 0);
          const uint32_t dA = smem_u32(sA + stage * C::A_BYTES), dB = smem_u32(sB + stage * C::B_BYTES);
          if (leader) mbar_expect_tx(fb, 2 * C::STAGE);
          if (p.a_mn) {
            tma_load_2d_pair(dA, &tmA, arow, kb * BK, bar);
            tma_load_2d_pair(dA + 8192, &tmA, arow + 64, kb * BK, bar);
          } else {
            tma_load_2d_pair(dA, &tmA, kb * BK, arow, bar);
          }
          if (p.b_mn) {
#pragma unroll
            for (int b = 0; b < BN / 128; ++b)
              tma_load_2d_pair(dB + b * 8192, &tmB, brow + 64 * b, kb * BK, bar);
          } else {
            tma_load_2d_pair(dB, &tmB, kb * BK, brow, bar);
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      const uint32_t idesc = idesc_bf16(2 * BM, BN) | (p.a_mn ? 1u << 15 : 0u) | (p.b_mn ? 1u << 16 : 0u);
      // descriptors of stage 0; a stage and a K step of 16 advance the address field (16-byte
      // units): 32 bytes along a swizzled row (K-major), 16 K rows of 128 bytes (MN-major)
      const uint64_t ad0 = p.a_mn ? mn_sw128_desc(smem_u32(sA)) : sw128_desc(smem_u32(sA));
      const uint64_t bd0 = p.b_mn ? mn_sw128_desc(smem_u32(sB)) : sw128_desc(smem_u32(sB));
      const uint32_t astep = p.a_mn ? 128 : 2, bstep = p.b_mn ? 128 : 2;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int i = 0;
      for (int t = unit; t < total && ok; t += units, ++i) {
        const int acc = i & 1;
        const uint32_t use = uint32_t(i >> 1) & 1u;
        ok = __all_sync(0xffffffffu, wait_bounded(tempty0 + 8 * acc, use ^ 1u, s_abort, p.status, wlimit));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + uint32_t(acc * BN);
        for (int kb = 0; kb < p.nkb; ++kb) {
          ok = __all_sync(0xffffffffu, wait_bounded(full0 + 8 * stage, phase, s_abort, p.status, wlimit));
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t ad = ad0 + uint64_t(stage * (C::A_BYTES >> 4));
            const uint64_t bd = bd0 + uint64_t(stage * (C::B_BYTES >> 4));
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_bf16_pair(d, ad + kk * astep, bd + kk * bstep, idesc, (kb | kk) != 0 ? 1u : 0u);
            mma_commit_pair(empty0 + 8 * stage, uint16_t(3));
          }
          __syncwarp();
          mma_any = true;
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok && lane == 0) mma_commit_pair(tfull0 + 8 * acc, uint16_t(3));
        __syncwarp();
      }
      if (!ok && mma_any && lane == 0) {  // every MMA issued must finish before TMEM is freed
        mma_commit_pair(drain_bar, uint16_t(1));
        wait_drain(drain_bar, 0u);
      }
      mma_drained = !ok && mma_any;
      __syncwarp();
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tempty_leader = cluster_addr(tempty0, 0);
    uint8_t* box = sBox + (warp - 2) * 4096;
    int nb = 0;  // the box of the next 32 columns
    int i = 0;
    // v (this lane's row, 32 columns) into box nb and out; the box's last store has been read
    auto write_box = [&](const CUtensorMap* map, const float (&v)[32], int col, int row) {
      uint8_t* b = box + nb * 2048;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(b + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(pack_bf16x2(v[8 * c], v[8 * c + 1]), pack_bf16x2(v[8 * c + 2], v[8 * c + 3]),
                       pack_bf16x2(v[8 * c + 4], v[8 * c + 5]), pack_bf16x2(v[8 * c + 6], v[8 * c + 7]));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (p.stream) tma_store_2d_hint(map, col, row, smem_u32(b), policy_evict_first());
        else tma_store_2d(map, col, row, smem_u32(b));
        bulk_commit();
      }
      nb ^= 1;
    };
    auto put = [&](const CUtensorMap* map, const float (&v)[32], int col, int row) {
      if (lane == 0) bulk_wait_read<1>();  // the store that last used this box has read it
      __syncwarp();
      write_box(map, v, col, row);
    };
    // res_tma: the residual's 32 x 32 box is brought into the box that the sum will leave from, a
    // step ahead (into box `b`, once every store so far has been read)
    const uint32_t res_bar = res0 + 16 * uint32_t(warp - 2);
    uint32_t res_phase = 0;  // bit b: phase of box b's barrier
    bool res_open = false;   // a box has been asked for and not waited for
    auto fetch_res = [&](int b, int col, int row) {
      if (lane == 0) {
        bulk_wait_read<0>();
        mbar_expect_tx(res_bar + 8 * b, 2048);
        tma_load_2d(smem_u32(box + b * 2048), &tmR, col, row, res_bar + 8 * b);
      }
      __syncwarp();
      res_open = true;
    };
    for (int t = unit; t < total; t += units, ++i) {
      const int acc = i & 1;
      const uint32_t use = uint32_t(i >> 1) & 1u;
      int m, n;
      decode(t, m, n);
      const int row0 = m * 2 * BM + int(rank) * BM + 32 * q, row = row0 + lane;
      const int cb = half * (BN / 2);
      const bool rows_here = row0 < p.rows;
      const int tile_col = n * BN;
      const __nv_bfloat16* rp = static_cast<const __nv_bfloat16*>(p.e.res) + row * p.e.ldr;
      if (p.res_tma && rows_here && tile_col + cb < p.cols) fetch_res(nb, tile_col + cb, row0);
      const bool ok = __all_sync(0xffffffffu, wait_bounded(tfull0 + 8 * acc, use, s_abort, p.status, wlimit));
      if (!ok) break;
      tc_fence_after();
      const uint32_t tbase = tmem + (uint32_t(q * 32) << 16) + uint32_t(acc * BN);
      bool landed = true;
#pragma unroll 1
      for (int c0 = cb; c0 < cb + BN / 2; c0 += 32) {
        const int col = tile_col + c0;
        if (!rows_here || col >= p.cols) break;  // warp-uniform: nothing of this part exists
        uint32_t acc32[32];
        tmem_ld16(tbase + c0, *reinterpret_cast<uint32_t(*)[16]>(acc32));
        tmem_ld16(tbase + c0 + 16, *reinterpret_cast<uint32_t(*)[16]>(acc32 + 16));
        uint4 rv[4];
        const bool rvec = !p.res_tma && p.res_vec && row < p.rows && col + 32 <= p.cols;
        if (p.res_tma) {
          landed = __all_sync(0xffffffffu, wait_bounded(res_bar + 8 * nb, (res_phase >> nb) & 1u, s_abort,
                                                        p.status, wlimit));
          if (!landed) {
            tmem_ld_wait();
            break;
          }
          res_phase ^= 1u << nb;
          res_open = false;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            rv[c] = *reinterpret_cast<const uint4*>(box + nb * 2048 + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4));
          if (c0 + 32 < cb + BN / 2 && col + 32 < p.cols) fetch_res(nb ^ 1, col + 32, row0);
        } else if (rvec) {
#pragma unroll
          for (int c = 0; c < 4; ++c) rv[c] = *reinterpret_cast<const uint4*>(rp + col + 8 * c);
        }
        float4 bv[8];  // the columns' biases, one address for the whole warp
        const bool bvec = p.bias_vec && col + 32 <= p.cols;
        if (bvec) {
#pragma unroll
          for (int j = 0; j < 8; ++j) bv[j] = __ldg(reinterpret_cast<const float4*>(p.e.bias + col) + j);
        }
        tmem_ld_wait();
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(acc32[j]);
        if (bvec) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 lo = unpack2(add2(pack2(v[4 * j], v[4 * j + 1]), pack2(bv[j].x, bv[j].y)));
            const float2 hi = unpack2(add2(pack2(v[4 * j + 2], v[4 * j + 3]), pack2(bv[j].z, bv[j].w)));
            v[4 * j] = lo.x; v[4 * j + 1] = lo.y; v[4 * j + 2] = hi.x; v[4 * j + 3] = hi.y;
          }
        } else if (p.e.bias) {
          const float bias = col + lane < p.cols ? __ldg(p.e.bias + col + lane) : 0.f;
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, bias, j);
        }
        if (p.e.pre) put(&tmP, v, col, row0);
        act_fast_all(p.e.act, v);
        if (rvec || p.res_tma) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t w[4] = {rv[c].x, rv[c].y, rv[c].z, rv[c].w};
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[h]));
              v[8 * c + 2 * h] += f.x;
              v[8 * c + 2 * h + 1] += f.y;
            }
          }
        } else if (p.e.res && row < p.rows) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (col + j < p.cols) v[j] += __bfloat162float(rp[col + j]);
        }
        if (p.res_tma) write_box(&tmY, v, col, row0);
        else put(&tmY, v, col, row0);
      }
      if (!landed) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + 8 * acc);
    }
    if (lane == 0) {  // the boxes are read, and a box asked for has landed, before they go away
      bulk_wait_all();
      if (res_open) {
        const int b = nb;  // before a tile: this box; inside one: the next
        wait_drain(res_bar + 8 * b, (res_phase >> b) & 1u);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0 && lane == 0) {
    const uint32_t peer = cluster_addr(smem_u32(const_cast<uint32_t*>(s_peer)), rank ^ 1u);
    st_cluster_u32(peer, issued);
    st_cluster_u32(peer + 4, uint32_t(*s_abort));
  }
  __syncwarp();
  cluster_sync_all();  // both CTAs done with TMEM and each other's barriers
  if (*s_abort || s_peer[1]) {
    // One CTA gave up: loads issued land and MMAs issued finish before shared and tensor memory
    // go away. The CTAs' producers are at most a use of each stage apart; the even CTA's full
    // barriers count both CTAs' bytes, so for a k-block that only one of them loaded the other's
    // part is settled first (its bytes taken as come, or the arrival that it would have made).
    if (warp == 0 && leader && lane == 0) {
      const uint32_t theirs = s_peer[0], lo = min(issued, theirs), hi = max(issued, theirs);
      for (uint32_t j = lo; j < hi; ++j) {
        const uint32_t fb = full0 + 8 * (j % C::STAGES);
        if (issued > theirs) mbar_complete_tx(fb, C::STAGE);
        else mbar_expect_tx(fb, C::STAGE);
      }
      for (uint32_t j = hi > C::STAGES ? hi - C::STAGES : 0; j < hi; ++j)
        wait_drain(full0 + 8 * (j % C::STAGES), (j / C::STAGES) & 1u);
    }
    if (warp == 1 && leader && lane == 0 && mma_any && !mma_drained) {
      mma_commit_pair(drain_bar, uint16_t(1));
      wait_drain(drain_bar, 0u);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::TMEM_COLS);
  }
}

bool out_aligned(const void* p, int64_t ld) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0);
}

template <int BN>
int run_pair(const LinearOperand& A, const LinearOperand& B, int rows, int cols, int K, const LinearEpi& e,
             unsigned* status, cudaStream_t st) {
  using C = PairCfg<BN>;
  CUtensorMap ta, tb, ty, tp, tr;
  int rc;
  if ((rc = map_operand(&ta, A, rows, K, BM)) != MOE_OK) return rc;
  if ((rc = map_operand(&tb, B, cols, K, BN / 2)) != MOE_OK) return rc;
  if ((rc = make_tma_map_out32(&ty, e.out, rows, cols, e.ldo)) != MOE_OK) return rc;
  tp = tr = ty;
  const bool res_tma = e.res && !e.pre && out_aligned(e.res, e.ldr);
  if (res_tma && (rc = make_tma_map_out32(&tr, const_cast<void*>(e.res), rows, cols, e.ldr)) != MOE_OK) return rc;
  if (e.pre && (rc = make_tma_map_out32(&tp, e.pre, rows, cols, e.ldp)) != MOE_OK) return rc;
  PairArgs p;
  p.rows = rows; p.cols = cols;
  p.nkb = (K + BK - 1) / BK;
  p.tiles_m = (rows + 2 * BM - 1) / (2 * BM);
  p.tiles_n = (cols + BN - 1) / BN;
  if (int64_t(p.tiles_m) * p.tiles_n > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  p.a_mn = A.mn; p.b_mn = B.mn;
  p.res_vec = e.res && out_aligned(e.res, e.ldr);
  p.res_tma = res_tma;
  p.bias_vec = e.bias && reinterpret_cast<uintptr_t>(e.bias) % 16 == 0;
  p.stream = int64_t(rows) * cols * 2 * (e.pre ? 2 : 1) > (int64_t(96) << 20);
  p.e = e;
  p.status = status;
  auto kern = linear_pair_kernel<BN>;
  static std::atomic<unsigned long long> seen{0};
  if ((rc = allow_smem(reinterpret_cast<const void*>(kern), C::SMEM, seen)) != MOE_OK) return rc;
  cudaLaunchConfig_t lc = {};
  lc.blockDim = dim3(kPairThreads);
  lc.dynamicSmemBytes = C::SMEM;
  lc.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  lc.gridDim = dim3(2);
  static std::atomic<int> resident{0};  // clusters the GPU holds at once (one kind of GPU)
  int clusters = resident.load(std::memory_order_relaxed);
  if (clusters == 0) {
    if (cudaOccupancyMaxActiveClusters(&clusters, kern, &lc) != cudaSuccess || clusters < 1)
      clusters = num_sms() / 2;
    resident.store(clusters, std::memory_order_relaxed);
  }
  lc.gridDim = dim3(unsigned(2 * std::min(clusters, p.tiles_m * p.tiles_n)));
  if (pdl_enabled()) {
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    lc.numAttrs = 2;
  }
  MOE_CUDA_CHECK(cudaLaunchKernelEx(&lc, kern, ta, tb, ty, tp, tr, p));
  return MOE_OK;
}

// K splits for `tiles` tiles: the largest power of two (at most 8, the portable cluster) whose
// CTAs all run at once, one an SM, with four k-blocks each at least. Clusters of 8 find room on 16 of
// the 18 to 20 SMs of a GPC; a second wave of clusters costs more than it saves (777 x 1408 x 1024:
// 84 tiles in 8 splits 24 us, unsplit 14 us).
int pick_splits(int64_t tiles, int K) {
  const int nkb = (K + BK - 1) / BK, room = num_sms() * 7 / 8;
  int s = 1;
  while (s < 8 && tiles * s * 2 <= room && nkb >= 8 * s) s *= 2;
  return s;
}

}  // namespace

int launch_linear_bf16(const LinearOperand& A, const LinearOperand& B, int rows, int cols, int K,
                       const LinearEpi& e, unsigned* status, cudaStream_t st) {
  const int64_t wide = (int64_t(cols) + BM - 1) / BM;
  if (rows <= 64 && !A.mn) {  // few rows: the wide side becomes the MMA's 128 rows
    const int s = pick_splits(wide, K);
    if (rows <= 16) return run_tile<16, true>(B, A, cols, rows, K, s, e, status, st);
    if (rows <= 32) return run_tile<32, true>(B, A, cols, rows, K, s, e, status, st);
    return run_tile<64, true>(B, A, cols, rows, K, s, e, status, st);
  }
  // 256-wide pair tiles once they fill the SM pairs; their outputs leave by TMA stores, which
  // need 16-byte rows
  const int64_t pairs = ((int64_t(rows) + 255) / 256) * ((int64_t(cols) + 255) / 256);
  if (pairs * 2 >= num_sms() / 2 && cols >= 128 && out_aligned(e.out, e.ldo) && out_aligned(e.pre, e.ldp))
    return run_pair<256>(A, B, rows, cols, K, e, status, st);
  const int64_t tiles = wide * ((int64_t(rows) + BM - 1) / BM);
  return run_tile<128, false>(A, B, rows, cols, K, pick_splits(tiles, K), e, status, st);
}

}  // namespace moe
