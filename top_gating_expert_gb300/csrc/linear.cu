// The linear layer y = act(x W^T + bias) + residual and its backward: argument checks, the
// workspace, the activation's derivative with the bias's gradient, and the copies of bf16
// operands that TMA cannot read in place. The products are in linear_bf16.cu and
// linear_f32.cu.
#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace {

constexpr int kColThreads = 32, kRowLanes = 8;

// d = dy act'(pre) (written to d when it is given) and the partial column sums of the
// unrounded d over a slice of rows: part[slice][N]. CTA: 32 threads of VEC columns by 8 row
// lanes; the lanes' sums are added in order. 16384 x 4096 bf16, gelu: 76 us for 403 MB (0.78 of the
// copy rate); four rows in flight a lane instead of two cost registers and 15 us.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kColThreads * kRowLanes)
    linear_dact_kernel(const T* __restrict__ dy, int64_t ldy, const T* __restrict__ pre, int64_t ldp,
                       T* __restrict__ d, int64_t ldd, int rows, int N, int slice, float* __restrict__ part) {
  __shared__ float s_sum[kRowLanes][kColThreads * VEC];
  pdl_wait();
  pdl_trigger();
  const int cx = threadIdx.x % kColThreads, ry = threadIdx.x / kColThreads;
  const int c = (blockIdx.x * kColThreads + cx) * VEC;
  const int64_t r0 = int64_t(blockIdx.y) * slice, r1 = min(int64_t(rows), r0 + slice);
  float acc[VEC];
#pragma unroll
  for (int q = 0; q < VEC; ++q) acc[q] = 0.f;
  if (c < N) {
#pragma unroll 2
    for (int64_t r = r0 + ry; r < r1; r += kRowLanes) {
      const Vec<T, VEC> g = load_vec<T, VEC>(dy + r * ldy + c);
      Vec<T, VEC> o, w;
      if constexpr (ACT != MOE_LIN_NONE) w = load_vec<T, VEC>(pre + r * ldp + c);
      if constexpr (sizeof(T) == 2 && VEC > 1 && ACT != MOE_LIN_NONE) {
#pragma unroll
        for (int q = 0; q < VEC; q += 2) {
          const f32x2 sl = slope_fast2<ACT>(pack2(to_f32(w.v[q]), to_f32(w.v[q + 1])));
          const f32x2 v = mul2(pack2(to_f32(g.v[q]), to_f32(g.v[q + 1])), sl);
          const float2 f = unpack2(v);
          acc[q] += f.x;
          acc[q + 1] += f.y;
          o.v[q] = from_f32<T>(f.x);
          o.v[q + 1] = from_f32<T>(f.y);
        }
      } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
          float v = to_f32(g.v[q]);
          if constexpr (ACT != MOE_LIN_NONE) {
            const float p = to_f32(w.v[q]);
            v *= sizeof(T) == 2 ? unpack2(slope_fast2<ACT>(pack2(p, p))).x : act_slope<ACT>(p);
          }
          acc[q] += v;
          o.v[q] = from_f32<T>(v);
        }
      }
      if (d) store_vec<T, VEC>(d + r * ldd + c, o);
    }
  }
  if (!part) return;
#pragma unroll
  for (int q = 0; q < VEC; ++q) s_sum[ry][cx * VEC + q] = acc[q];
  __syncthreads();
  for (int x = threadIdx.x; x < kColThreads * VEC; x += kColThreads * kRowLanes) {
    const int cc = blockIdx.x * kColThreads * VEC + x;
    if (cc >= N) continue;
    float s = 0.f;
#pragma unroll
    for (int l = 0; l < kRowLanes; ++l) s += s_sum[l][x];
    part[int64_t(blockIdx.y) * N + cc] = s;
  }
}

// out[c] = sum over the slices of part[s][c]
__global__ void __launch_bounds__(1024)
    linear_dbias_kernel(const float* __restrict__ part, int slices, int N, float* __restrict__ out) {
  __shared__ float s_part[32][33];
  pdl_wait();
  pdl_trigger();
  column_sums(slices, blockIdx.x * 32, N, s_part, [&](int s, int c) { return part[int64_t(s) * N + c]; },
              [&](int c, float t) { out[c] = t; });
}

// Copies of up to two operands to 16-byte rows: dst [rows][ldd] = src [rows][cols], src on any
// element boundary. Eight elements a thread, read as the 4-byte words that hold them (five when
// the row starts inside a word) and shifted into place; a word that the row only half fills is read
// as its one element, so nothing outside of the row is read. A warp takes 256 columns of a row.
struct AlignJob {
  const __nv_bfloat16* src;
  int64_t ld, rows;
  int cols;
  __nv_bfloat16* dst;
  int64_t ldd;
};

__global__ void __launch_bounds__(256) linear_align_kernel(AlignJob j0, AlignJob j1) {
  pdl_wait();
  pdl_trigger();
  const AlignJob j = blockIdx.y ? j1 : j0;
  const int per = int(j.ldd / 8), lane = threadIdx.x & 31;
  for (int64_t r = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); r < j.rows; r += int64_t(gridDim.x) * 8) {
    const uintptr_t row = reinterpret_cast<uintptr_t>(j.src + r * j.ld);
    const int odd = int(row >> 1) & 1;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(row & ~uintptr_t(3));
    for (int p = blockIdx.z * 32 + lane; p < per; p += gridDim.z * 32) {
      const int left = j.cols - 8 * p;  // >= 1
      const uint32_t* w = words + 4 * p;
      uint32_t v[5];
#pragma unroll
      for (int q = 0; q < 5; ++q) {
        const int at = 2 * q - odd;  // the word's first element, from this thread's first one on
        const bool head = at < 0 && p == 0, tail = at + 1 >= left;
        const uint16_t* one = reinterpret_cast<const uint16_t*>(w + q);
        v[q] = 0u;
        if (at < left && (q < 4 || odd)) {
          if (head) v[q] = uint32_t(__ldg(one + 1)) << 16;
          else if (tail) v[q] = __ldg(one);
          else v[q] = __ldg(w + q);
        }
      }
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = odd ? __funnelshift_r(v[q], v[q + 1], 16) : v[q];
      *reinterpret_cast<uint4*>(j.dst + r * j.ldd + 8 * p) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

int64_t up8(int64_t x) { return (x + 7) / 8 * 8; }

// slices of the bias's gradient: about 1216 CTAs of 256 columns (eight an SM) at most
int bias_slices(int T, int N) {
  const int cblocks = (N + 255) / 256;
  const int s = std::max(1, std::min(256, 1216 / cblocks));
  return std::max(1, std::min(s, (T + 4 * kRowLanes - 1) / (4 * kRowLanes)));  // four rows a lane
}

int check_linear(const moe_linear_t* p, moe_linear_t* q) {
  if (!p || p->T < 0 || p->N < 1 || p->K < 1) return MOE_ERR_INVALID_ARG;
  if (p->act < MOE_LIN_NONE || p->act > MOE_LIN_SILU) return MOE_ERR_INVALID_ARG;
  if (p->dtype != MOE_F32 && p->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (p->T > (1 << 30) || p->N > (1 << 22) || p->K > (1 << 22)) return MOE_ERR_UNSUPPORTED;
  *q = *p;
  auto ld = [](int64_t& v, int64_t n) {
    if (v == 0) v = n;
    return v >= n;
  };
  if (!ld(q->ldx, p->K) || !ld(q->ldw, p->K) || !ld(q->ldy, p->N) || !ld(q->ldr, p->N) ||
      !ld(q->ldp, p->N) || !ld(q->lddx, p->K) || !ld(q->lddw, p->K))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Carves the workspace: regions in a fixed order, their total compared with what there is.
struct Carver {
  char* base;
  size_t at = 256;
  void* take(size_t bytes) {
    void* p = base ? base + at : nullptr;
    at = align256(at + bytes);
    return p;
  }
};

// Few tokens forward: W is streamed row by row, nothing copied and no partial sums.
bool few_tokens(const moe_linear_t& p) { return p.T <= (p.dtype == MOE_BF16 ? 1 : 8); }

size_t ws_need(const moe_linear_t& p, bool backward, bool all) {
  Carver c{nullptr};
  if (!backward && few_tokens(p)) return c.at;
  const int64_t Kp = up8(p.K), Np = up8(p.N);
  if (p.dtype == MOE_F32) {
    c.take(kPartBytes);
    if (backward && p.act != MOE_LIN_NONE) c.take(size_t(p.T) * Np * 4);
  } else {
    if (all || p.ldx % 8) c.take(size_t(p.T) * Kp * 2);
    if (all || p.ldw % 8) c.take(size_t(p.N) * Kp * 2);
    if (backward && (all || p.act != MOE_LIN_NONE || p.ldy % 8)) c.take(size_t(p.T) * Np * 2);
  }
  if (backward) c.take(size_t(bias_slices(p.T, p.N)) * p.N * 4);
  return c.at;
}

bool in_place(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; }

// The operand [rows, cols] as TMA can read it: in place, or in a copy with 16-byte rows that the
// job describes (src null: none).
int align_operand(const void* src, int64_t ld, int64_t rows, int cols, Carver& c, size_t ws_bytes,
                  LinearOperand* o, AlignJob* job) {
  o->p = src;
  o->ld = ld;
  *job = AlignJob{nullptr, 0, 0, 1, nullptr, 8};
  if (in_place(src, ld)) return MOE_OK;
  o->ld = up8(cols);
  void* dst = c.take(size_t(rows) * o->ld * 2);
  o->p = dst;
  *job = AlignJob{static_cast<const __nv_bfloat16*>(src), ld, rows, cols, static_cast<__nv_bfloat16*>(dst), o->ld};
  return c.at > ws_bytes ? MOE_ERR_WORKSPACE : MOE_OK;
}

int launch_align(const AlignJob& a, const AlignJob& b, cudaStream_t st) {
  const bool two = a.src && b.src;
  if (!a.src && !b.src) return MOE_OK;
  const AlignJob& one = a.src ? a : b;
  const int64_t rows = std::max(one.rows, two ? b.rows : 0), per = std::max(one.ldd, two ? b.ldd : 0) / 8;
  const dim3 grid(unsigned(std::min<int64_t>((rows + 7) / 8, 1 << 20)), two ? 2 : 1,
                  unsigned(std::min<int64_t>((per + 31) / 32, 64)));
  return launch_kernel(linear_align_kernel, grid, dim3(256), 0, st, one, b);
}

// d (when it is given) and dbias (when it is given; part: its slices' partial sums)
template <typename T>
int launch_dact(const moe_linear_t& p, const void* dy, const void* pre, void* d, int64_t ldd, float* part,
                float* dbias, cudaStream_t st) {
  if (!d && !dbias) return MOE_OK;
  constexpr int V = 16 / int(sizeof(T));
  auto ok = [](const void* q, int64_t ld) {
    return !q || (reinterpret_cast<uintptr_t>(q) % 16 == 0 && ld % V == 0);
  };
  const bool vec = p.N % V == 0 && ok(dy, p.ldy) && ok(pre, p.ldp) && ok(d, ldd);
  const int slices = bias_slices(p.T, p.N), slice = (p.T + slices - 1) / slices;
  float* sums = dbias ? (slices == 1 ? dbias : part) : nullptr;  // one slice: the sum itself
  const int rc = with_act(p.act, [&](auto tag) {
    constexpr int ACT = decltype(tag)::value;
    const int cols = kColThreads * (vec ? V : 1);
    auto kern = vec ? linear_dact_kernel<T, V, ACT> : linear_dact_kernel<T, 1, ACT>;
    return launch_kernel(kern, dim3(unsigned((p.N + cols - 1) / cols), unsigned(slices)),
                         dim3(kColThreads * kRowLanes), 0, st, static_cast<const T*>(dy), p.ldy,
                         static_cast<const T*>(pre), p.ldp, static_cast<T*>(d), ldd, p.T, p.N, slice, sums);
  });
  if (rc != MOE_OK || !dbias || slices == 1) return rc;
  return launch_kernel(linear_dbias_kernel, dim3(unsigned((p.N + 31) / 32)), dim3(1024), 0, st,
                       static_cast<const float*>(part), slices, p.N, dbias);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_linear_workspace_bytes(const moe_linear_t* p, int backward, int unaligned, size_t* bytes) {
  moe_linear_t q;
  const int rc = check_linear(p, &q);
  if (rc != MOE_OK) return rc;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = ws_need(q, backward != 0, unaligned != 0);
  return MOE_OK;
}

int moe_linear_forward(const moe_linear_t* p, const void* x, const void* W, const float* bias,
                       const void* residual, void* y, void* pre, void* ws, size_t ws_bytes,
                       moe_stream_t stream) {
  moe_linear_t q;
  int rc = check_linear(p, &q);
  if (rc != MOE_OK) return rc;
  if (q.T == 0) return MOE_OK;
  if (!x || !W || !y || (pre && pre == y)) return MOE_ERR_INVALID_ARG;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < ws_need(q, false, false))
    return MOE_ERR_WORKSPACE;
  LinearEpi e;
  e.bias = bias; e.res = residual; e.out = y; e.pre = pre;
  e.ldo = q.ldy; e.ldr = q.ldr; e.ldp = q.ldp;
  e.act = q.act;
  if (few_tokens(q))
    return launch_linear_few(q.dtype == MOE_BF16, x, q.ldx, W, q.ldw, q.T, q.N, q.K, e, stream);
  Carver c{static_cast<char*>(ws)};
  if (q.dtype == MOE_F32) {
    float* part = static_cast<float*>(c.take(kPartBytes));
    return launch_linear_f32(static_cast<const float*>(x), q.ldx, 1, static_cast<const float*>(W), q.ldw,
                             1, q.T, q.N, q.K, e, part, stream);
  }
  LinearOperand a{nullptr, 0, false}, b{nullptr, 0, false};
  AlignJob ja, jb;
  if ((rc = align_operand(x, q.ldx, q.T, q.K, c, ws_bytes, &a, &ja)) != MOE_OK ||
      (rc = align_operand(W, q.ldw, q.N, q.K, c, ws_bytes, &b, &jb)) != MOE_OK ||
      (rc = launch_align(ja, jb, stream)) != MOE_OK)
    return rc;
  return launch_linear_bf16(a, b, q.T, q.N, q.K, e, static_cast<unsigned*>(ws), stream);
}

int moe_linear_backward(const moe_linear_t* p, const void* dy, const void* x, const void* W,
                        const void* pre, void* dx, void* dW, float* dbias, void* ws,
                        size_t ws_bytes, moe_stream_t stream) {
  moe_linear_t q;
  int rc = check_linear(p, &q);
  if (rc != MOE_OK) return rc;
  const size_t eb = q.dtype == MOE_BF16 ? 2 : 4;
  if (q.T == 0) {
    if (dW) MOE_CUDA_CHECK(cudaMemset2DAsync(dW, size_t(q.lddw) * eb, 0, size_t(q.K) * eb, size_t(q.N), stream));
    if (dbias) MOE_CUDA_CHECK(cudaMemsetAsync(dbias, 0, size_t(q.N) * 4, stream));
    return MOE_OK;
  }
  if (!dy || (dx && !W) || (dW && !x) || (q.act != MOE_LIN_NONE && !pre)) return MOE_ERR_INVALID_ARG;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < ws_need(q, true, false))
    return MOE_ERR_WORKSPACE;
  if (q.act == MOE_LIN_NONE) pre = nullptr;
  const int64_t Np = up8(q.N);
  Carver c{static_cast<char*>(ws)};
  if (q.dtype == MOE_F32) {
    float* part = static_cast<float*>(c.take(kPartBytes));
    void* d = pre ? c.take(size_t(q.T) * Np * 4) : nullptr;
    float* dbp = static_cast<float*>(c.take(size_t(bias_slices(q.T, q.N)) * q.N * 4));
    if ((rc = launch_dact<float>(q, dy, pre, d, Np, dbp, dbias, stream)) != MOE_OK) return rc;
    const float* df = static_cast<const float*>(pre ? d : dy);
    const int64_t ldd = pre ? Np : q.ldy;
    LinearEpi e;
    if (dx) {
      e.out = dx; e.ldo = q.lddx;
      if ((rc = launch_linear_f32(df, ldd, 1, static_cast<const float*>(W), 1, q.ldw, q.T, q.K, q.N, e,
                                  part, stream)) != MOE_OK)
        return rc;
    }
    if (dW) {
      e.out = dW; e.ldo = q.lddw;
      return launch_linear_f32(df, 1, ldd, static_cast<const float*>(x), 1, q.ldx, q.N, q.K, q.T, e, part,
                               stream);
    }
    return MOE_OK;
  }
  const bool make_d = pre || !in_place(dy, q.ldy);  // d written out: the products' operand
  LinearOperand xo{nullptr, 0, true}, wo{nullptr, 0, true};
  void* d = nullptr;
  float* dbp = nullptr;
  AlignJob jx{nullptr, 0, 0, 1, nullptr, 8}, jw = jx;
  if (dW && (rc = align_operand(x, q.ldx, q.T, q.K, c, ws_bytes, &xo, &jx)) != MOE_OK) return rc;
  if (dx && (rc = align_operand(W, q.ldw, q.N, q.K, c, ws_bytes, &wo, &jw)) != MOE_OK) return rc;
  if (make_d) d = c.take(size_t(q.T) * Np * 2);
  dbp = static_cast<float*>(c.take(size_t(bias_slices(q.T, q.N)) * q.N * 4));
  if (c.at > ws_bytes) return MOE_ERR_WORKSPACE;
  if ((rc = launch_align(jx, jw, stream)) != MOE_OK) return rc;
  if ((rc = launch_dact<__nv_bfloat16>(q, dy, pre, d, Np, dbp, dbias, stream)) != MOE_OK) return rc;
  LinearOperand dk{make_d ? d : dy, make_d ? Np : q.ldy, false};
  unsigned* status = static_cast<unsigned*>(ws);
  LinearEpi e;
  if (dx) {  // d W: W's rows run along the reduction, so it is read MN-major
    e.out = dx; e.ldo = q.lddx;
    if ((rc = launch_linear_bf16(dk, wo, q.T, q.K, q.N, e, status, stream)) != MOE_OK) return rc;
  }
  if (dW) {  // d^T x: both operands' rows run along the reduction
    e.out = dW; e.ldo = q.lddw;
    dk.mn = true;
    return launch_linear_bf16(dk, xo, q.N, q.K, q.T, e, status, stream);
  }
  return MOE_OK;
}

}  // extern "C"
