// Cross entropy of a linear head over a large vocabulary, l = x W^T, without storing the logits:
// argument checks, workspace, the order of the products (linear_bf16.cuh, linear_f32.cu) and the
// kernels that join their results.
//
//   loss = lse - l[target] + z lse^2,   d = w ((1 + 2 z lse) exp(l - lse) - [target]),
//   dx = d W,   dW = d^T x
//
// Forward, bf16: one product whose epilogue keeps of 128 or 256 columns of a row their largest logit and sum
// of exponentials (8 bytes) and the target's logit; xent_join_kernel joins them.
// Backward, bf16: a piece of the vocabulary at a time, the logits once more, d in bf16 into the
// workspace, then its share of dx (fp32 sums over the pieces) and the rows of dW, which are whole. Pieces of
// about 512 MB of d: small enough for memory (the logits of 8192 tokens and 131072 entries take 4.3 GB in
// fp32). The sums' way through memory, 8 bytes an element of dx and piece, is about 350 / entries of the products'
// time, and a piece has 2^28 / tokens entries: 1 % at 8192 tokens, 2 at 16384, 9 at 65536 (65536 x 32768 x 1024: 8.2 to 8.9 ms,
// in one piece of 4.3 GB 8.1), 68 with the least piece, from half a million tokens on. Who has memory for larger
// pieces gives their size.
// d of the mean loss is kept without the weight that all tokens share, which the products' results take:
// rounding to bf16 then leaves the target's entry, near -1, almost as it is, where w (p - 1) would be off by up to
// 2^-8, the same way in every token (8192 x 65536 x 2048: gradients 3.1e-3 off in all with w in d, now 1.7e-3,
// their own rounding; with 64 entries and fewer d's rounding makes it 2.0e-3 to 2.5e-3).
// fp32: the logits of a piece go through the workspace; the plain-FMA products are by far the longest part.
// Measured: 8192 x 65536 x 2048 forward 1.12 ms, backward 3.9 (tensor pipe 83 to 90 % active); 8192 x 32768 x 1024
// forward 303 us, backward 962; 1 x 32768 x 1024 forward 26 us alone. The tensor cores' sums truncate: lse comes
// out low by 3e-7 of itself for every 1024 of K.
#include <math.h>

#include <algorithm>

#include "linear.cuh"

namespace moe {
namespace {

constexpr float kL2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
constexpr size_t kPieceBytes = size_t(512) << 20;  // of d (bf16) or logits (fp32)
constexpr size_t kStatBytes = size_t(256) << 20;   // of the forward's 8 bytes for 128 logits or more: tokens at a time
constexpr int kLeastPiece = 512;

// The join of n (c, s) pairs of 32 tokens: each of 32 warps every 32nd pair (a lane a token), then warp w joins
// token w's 32 results: lse, the token's loss, and the CTA's sum of losses and count of targets. The last
// CTA of the last launch sums those in order (fp64) into stats. NaN stays NaN; a pair of c = -inf has s = 0.
struct JoinArgs {
  const float2* part;
  int64_t ldpart;
  int n, rows, V;
  const float* hit;
  const int64_t* target;
  int64_t ignore;
  float z;
  float *loss, *lse, *stats;
  float2* sums;  // a CTA's, over all launches
  unsigned first, ctas;
  unsigned* status;
};
__device__ __forceinline__ void join_pair(float& c, float& s, float pc, float ps) {
  const float cn = fmaxf(c, pc), base = cn == -INFINITY ? 0.f : cn;
  s = s * exp2f(c - base) + ps * exp2f(pc - base);
  c = cn;
}

// sums over a warp, in every lane, in the order of a fixed tree
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__global__ void __launch_bounds__(1024) xent_join_kernel(const JoinArgs a) {
  __shared__ float2 s_part[32][33];
  __shared__ float s_loss[32];
  __shared__ int s_one[32];
  __shared__ double s_sum[32];
  __shared__ bool s_last;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * 32 + lane, row = blockIdx.x * 32 + warp;
  // for the end: this warp's token
  int64_t y = a.ignore;
  float hit = 0.f;
  if (row < a.rows) {
    y = __ldg(a.target + row);
    hit = __ldg(a.hit + row);  // any, without a target among the logits
  }
  float c = -INFINITY, s = 0.f;
  if (t < a.rows) {
    float2 p[8];  // eight pairs in flight
    for (int i0 = warp; i0 < a.n; i0 += 256) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (i0 + 32 * q < a.n) p[q] = __ldg(a.part + (i0 + 32 * q) * a.ldpart + t);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (i0 + 32 * q < a.n) join_pair(c, s, p[q].x, p[q].y);
    }
  }
  s_part[warp][lane] = make_float2(c, s);
  __syncthreads();
  const float2 p = s_part[lane][warp];
  float top = p.x;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  s = warp_sum(p.y * exp2f(p.x - (top == -INFINITY ? 0.f : top)));
  if (lane == 0) {
    float loss = 0.f;
    if (row < a.rows) {
      const float lse = (top + log2f(s)) * kLn2;
      if (y != a.ignore) {
        loss = lse - hit + a.z * lse * lse;
        if (y < 0 || y >= a.V) {
          loss = __int_as_float(0x7fc00000);
          atomicOr(a.status, kStatusDeviceData);
        }
      }
      a.lse[row] = lse;
      a.loss[row] = loss;
    }
    s_loss[warp] = loss;
    s_one[warp] = y != a.ignore;
  }
  __syncthreads();
  if (warp == 0) {
    const float sum = warp_sum(s_loss[lane]);
    const int cnt = __popc(__ballot_sync(0xffffffffu, s_one[lane] != 0));
    if (lane == 0 && a.ctas == 1) {
      a.stats[0] = cnt > 0 ? sum / float(cnt) : 0.f;
      a.stats[1] = float(cnt);
      s_last = false;
    } else if (lane == 0) {
      a.sums[a.first + blockIdx.x] = make_float2(sum, float(cnt));
      __threadfence();
      s_last = atomicAdd(a.status + 1, 1u) == a.ctas - 1;
    }
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double sum = 0.0;
  int cnt = 0;
  for (unsigned i = threadIdx.x; i < a.ctas; i += 1024) {
    const float2 b = __ldcg(a.sums + i);
    sum += double(b.x);
    cnt += int(b.y);
  }
  sum = warp_sum(sum);
  cnt = __reduce_add_sync(0xffffffffu, cnt);
  if (lane == 0) {
    s_sum[warp] = sum;
    s_one[warp] = cnt;
  }
  __syncthreads();
  if (warp == 0) {
    sum = warp_sum(s_sum[lane]);
    cnt = __reduce_add_sync(0xffffffffu, s_one[lane]);
    if (lane == 0) {
      a.stats[0] = cnt > 0 ? float(sum) / float(cnt) : 0.f;
      a.stats[1] = float(cnt);
      a.status[1] = 0u;  // the ticket
    }
  }
}

// fp32 logits of a piece [rows, cols] (row stride ld): the row's (c, s) and its target's logit.
__global__ void __launch_bounds__(256)
    xent_stats_f32_kernel(const float* __restrict__ l, int64_t ld, int cols, const int64_t* __restrict__ target, int v0,
                          float2* __restrict__ part, float* __restrict__ hit) {
  __shared__ float s_c[8], s_s[8];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const float* p = l + row * ld;
  float c = -INFINITY, s = 0.f;
  for (int i = threadIdx.x; i < cols; i += 1024) {
    float v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = i + 256 * q < cols ? p[i + 256 * q] : -INFINITY;
    const float cn = fmaxf(c, fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) * kL2e), base = cn == -INFINITY ? 0.f : cn;
    s *= exp2f(c - base);
#pragma unroll
    for (int q = 0; q < 4; ++q) s += exp2f(fmaf(v[q], kL2e, -base));
    c = cn;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float oc = __shfl_xor_sync(0xffffffffu, c, off), os = __shfl_xor_sync(0xffffffffu, s, off);
    join_pair(c, s, oc, os);
  }
  if (lane == 0) {
    s_c[warp] = c;
    s_s[warp] = s;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    c = s_c[0];
    s = s_s[0];
    for (int w = 1; w < 8; ++w) join_pair(c, s, s_c[w], s_s[w]);
    part[row] = make_float2(c, s);
    const int64_t y = target[row] - v0;
    if (y >= 0 && y < cols) hit[row] = p[y];
  }
}

// d in place of the fp32 logits of a piece.
__global__ void __launch_bounds__(256)
    xent_grad_f32_kernel(float* __restrict__ l, int64_t ld, int cols, const XentEpi x, unsigned* status) {
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  float4 r = xent_row(x, row);
  const float f = xent_factor(x);
  if (x.v0 == 0 && blockIdx.y == 0 && threadIdx.x == 0 && xent_bad_target(x, row)) atomicOr(status, kStatusDeviceData);
  const int at = __float_as_int(r.w) - x.v0;
  const bool on = r.z != 0.f;
  r.y *= f;
  r.z *= f;
  for (int i = blockIdx.y * 256 + threadIdx.x; i < cols; i += gridDim.y * 256) {
    float d = 0.f;
    if (on) {
      d = exp2f(fmaf(l[row * ld + i], kL2e, -r.x)) * r.y;
      if (i == at) d -= r.z;
    }
    l[row * ld + i] = d;
  }
}

int check_xent(const moe_xent_t* p, moe_xent_t* q) {
  if (!p || p->T < 0 || p->V < 1 || p->K < 1 || p->piece < 0) return MOE_ERR_INVALID_ARG;
  if (p->dtype != MOE_F32 && p->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (!(p->z_coef >= 0.f) || !std::isfinite(p->z_coef)) return MOE_ERR_INVALID_ARG;
  if (p->T > (1 << 30) || p->V > (1 << 22) || p->K > (1 << 22)) return MOE_ERR_UNSUPPORTED;
  *q = *p;
  auto ld = [](int64_t& v, int64_t n) {
    if (v == 0) v = n;
    return v >= n;
  };
  if (!ld(q->ldx, p->K) || !ld(q->ldw, p->K) || !ld(q->lddx, p->K) || !ld(q->lddw, p->K)) return MOE_ERR_INVALID_ARG;
  // pieces of about equal size, whole tiles where there are several
  int64_t v = p->piece ? p->piece
                       : int64_t(kPieceBytes / (size_t(std::max(1, p->T)) * (p->dtype == MOE_BF16 ? 2 : 4)));
  v = std::max<int64_t>(v, kLeastPiece);
  const int64_t n = (p->V + v - 1) / v;
  q->piece = n == 1 ? p->V : int(std::min<int64_t>(p->V, ((p->V + n - 1) / n + 255) / 256 * 256));
  return MOE_OK;
}

int pieces(const moe_xent_t& p) { return (p.V + p.piece - 1) / p.piece; }
int slots(const moe_xent_t& p) { return p.dtype == MOE_BF16 ? (p.V + 127) / 128 : pieces(p); }
// tokens of a forward product: as many as the room for its partial results holds
// (fp32: all of them, the logits of a piece take far more)
int forward_rows(const moe_xent_t& p) {
  if (p.dtype == MOE_F32) return std::max(1, p.T);
  const int64_t most = std::max<int64_t>(256, int64_t(kStatBytes / (size_t(slots(p)) * 8)) / 256 * 256);
  return int(std::min<int64_t>(std::max(1, p.T), most));
}

// parts of the reduction of dx over a piece (the last piece may be shorter: the same parts, if it has as many k-blocks)
int dx_splits(const moe_xent_t& p) { return p.T ? product_sum_splits(p.T, p.K, p.piece) : 1; }

// Regions behind the operands' copies; the forward's and the backward's share their room.
struct Regions {
  float2 *part = nullptr, *sums = nullptr;
  float* hit = nullptr;
  void* d = nullptr;  // [T][up8(piece)]: bf16 d, or fp32 logits
  float* acc = nullptr;
  float* split = nullptr;
  float* prod = nullptr;  // the fp32 products' partial sums
};
void carve(const moe_xent_t& p, bool backward, Carver& c, Regions* r) {
  const size_t T = size_t(std::max(1, p.T));
  const bool f32 = p.dtype == MOE_F32;
  if (f32) r->prod = static_cast<float*>(c.take(kPartBytes));
  if (f32 || backward) r->d = c.take(T * up8(p.piece) * (f32 ? 4 : 2));
  if (!backward) {
    r->part = static_cast<float2*>(c.take(size_t(slots(p)) * forward_rows(p) * 8));
    r->hit = static_cast<float*>(c.take(size_t(forward_rows(p)) * 4));
    r->sums = static_cast<float2*>(c.take((T + 31) / 32 * 8 + size_t((p.T + forward_rows(p) - 1) / forward_rows(p)) * 8));
  } else {
    if (!f32 && pieces(p) > 1) r->acc = static_cast<float*>(c.take(T * up8(p.K) * 4));
    const int n = f32 ? 1 : dx_splits(p);
    if (n > 1) r->split = static_cast<float*>(c.take(n * T * up8(p.K) * 4));
  }
}

size_t ws_need(const moe_xent_t& p, bool backward, bool all) {
  Carver c{nullptr};
  const int64_t Kp = up8(p.K);
  if (p.dtype == MOE_BF16) {
    if (all || p.ldx % 8) c.take(size_t(p.T) * Kp * 2);
    if (all || p.ldw % 8) c.take(size_t(p.V) * Kp * 2);
  }
  Regions r;
  Carver f = c, b = c;
  carve(p, false, f, &r);
  if (backward) carve(p, true, b, &r);
  return std::max(f.at, b.at);
}

// x and W as the products read them.
int operands(const moe_xent_t& p, const void* x, const void* W, Carver& c, size_t ws_bytes, LinearOperand* a,
             LinearOperand* b, cudaStream_t st) {
  *a = LinearOperand{x, p.ldx, false};
  *b = LinearOperand{W, p.ldw, false};
  if (p.dtype != MOE_BF16) return MOE_OK;
  AlignJob ja, jb;
  int rc;
  if ((rc = align_operand(x, p.ldx, p.T, p.K, c, ws_bytes, a, &ja)) != MOE_OK ||
      (rc = align_operand(W, p.ldw, p.V, p.K, c, ws_bytes, b, &jb)) != MOE_OK)
    return rc;
  return launch_align(ja, jb, st);
}

LinearOperand rows_from(const LinearOperand& o, int64_t r, size_t eb) {
  return LinearOperand{static_cast<const char*>(o.p) + r * o.ld * eb, o.ld, o.mn};
}

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  return !ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || ws_bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

// the fp32 logits of a piece into r.d
int logits_f32(const moe_xent_t& p, const LinearOperand& a, const LinearOperand& b, int v0, int nv, const Regions& r,
               cudaStream_t st) {
  LinearEpi e;
  e.out = r.d;
  e.ldo = up8(p.piece);
  return launch_linear_f32(static_cast<const float*>(a.p), a.ld, 1, static_cast<const float*>(b.p) + v0 * b.ld, b.ld, 1,
                           p.T, nv, p.K, e, r.prod, st);
}

int forward(const moe_xent_t& p, const void* x, const void* W, const int64_t* target, float* loss, float* lse,
            float* stats, void* ws, size_t ws_bytes, cudaStream_t st) {
  Carver c{static_cast<char*>(ws)};
  LinearOperand a, b;
  Regions r;
  int rc;
  // the workspace is checked against what these operands take before anything is launched
  Carver probe{nullptr};
  if (p.dtype == MOE_BF16) {
    if (p.ldx % 8 || reinterpret_cast<uintptr_t>(x) % 16) probe.take(size_t(p.T) * up8(p.K) * 2);
    if (p.ldw % 8 || reinterpret_cast<uintptr_t>(W) % 16) probe.take(size_t(p.V) * up8(p.K) * 2);
  }
  carve(p, false, probe, &r);
  if ((rc = check_ws(ws, ws_bytes, probe.at)) != MOE_OK) return rc;
  if ((rc = operands(p, x, W, c, ws_bytes, &a, &b, st)) != MOE_OK) return rc;
  carve(p, false, c, &r);
  unsigned* status = static_cast<unsigned*>(ws);
  const int step = forward_rows(p), f32 = p.dtype == MOE_F32;
  unsigned ctas = 0;
  for (int64_t t0 = 0; t0 < p.T; t0 += step) ctas += unsigned((std::min<int64_t>(step, p.T - t0) + 31) / 32);
  unsigned first = 0;
  if (f32) {  // the stats of all tokens, a piece after the other
    for (int v0 = 0, i = 0; v0 < p.V; v0 += p.piece, ++i) {
      const int nv = std::min(p.piece, p.V - v0);
      if ((rc = logits_f32(p, a, b, v0, nv, r, st)) != MOE_OK) return rc;
      if ((rc = launch_kernel(xent_stats_f32_kernel, dim3(unsigned(p.T)), dim3(256), 0, st,
                              static_cast<const float*>(r.d), up8(p.piece), nv, target, v0, r.part + i * int64_t(step),
                              r.hit)) != MOE_OK)
        return rc;
    }
  }
  for (int64_t t0 = 0; t0 < p.T; t0 += step) {
    const int rows = int(std::min<int64_t>(step, p.T - t0));
    if (!f32) {
      XentEpi e;
      e.part = r.part; e.ldpart = step; e.hit = r.hit; e.target = target + t0;
      if ((rc = launch_xent_bf16(kXentStats, rows_from(a, t0, 2), b, rows, p.V, p.K, LinearEpi{}, e, status, st)) !=
          MOE_OK)
        return rc;
    }
    JoinArgs j;
    const int w = f32 ? p.piece : xent_stats_cols(rows, p.V);
    j.part = r.part; j.ldpart = step; j.n = (p.V + w - 1) / w; j.rows = rows; j.V = p.V;
    j.hit = r.hit; j.target = target + t0; j.ignore = p.ignore_index; j.z = p.z_coef;
    j.loss = loss + t0; j.lse = lse + t0; j.stats = stats;
    j.sums = r.sums; j.first = first; j.ctas = ctas;
    j.status = status;
    const unsigned grid = unsigned((rows + 31) / 32);
    if ((rc = launch_kernel(xent_join_kernel, dim3(grid), dim3(1024), 0, st, j)) != MOE_OK) return rc;
    first += grid;
  }
  return MOE_OK;
}

int backward(const moe_xent_t& p, const void* x, const void* W, const int64_t* target, const float* lse,
             const float* dloss, const float* stats, float scale, void* dx, void* dW, void* ws, size_t ws_bytes,
             cudaStream_t st) {
  Carver c{static_cast<char*>(ws)};
  LinearOperand a, b;
  Regions r;
  int rc;
  Carver probe{nullptr};
  if (p.dtype == MOE_BF16) {
    if (p.ldx % 8 || reinterpret_cast<uintptr_t>(x) % 16) probe.take(size_t(p.T) * up8(p.K) * 2);
    if (p.ldw % 8 || reinterpret_cast<uintptr_t>(W) % 16) probe.take(size_t(p.V) * up8(p.K) * 2);
  }
  carve(p, true, probe, &r);
  if ((rc = check_ws(ws, ws_bytes, probe.at)) != MOE_OK) return rc;
  if ((rc = operands(p, x, W, c, ws_bytes, &a, &b, st)) != MOE_OK) return rc;
  carve(p, true, c, &r);
  unsigned* status = static_cast<unsigned*>(ws);
  const int64_t ldd = up8(p.piece);
  const bool f32 = p.dtype == MOE_F32;
  XentEpi g;  // what all pieces share
  g.target = target; g.lse = lse; g.dloss = dloss; g.ignore = p.ignore_index; g.z = p.z_coef; g.V = p.V;
  g.stats = dloss ? nullptr : stats;
  g.scale = scale;
  for (int v0 = 0; v0 < p.V; v0 += p.piece) {
    const int nv = std::min(p.piece, p.V - v0);
    const bool first = v0 == 0, last = v0 + nv == p.V;
    g.v0 = v0;
    if (f32) {
      if ((rc = logits_f32(p, a, b, v0, nv, r, st)) != MOE_OK) return rc;
      float* d = static_cast<float*>(r.d);
      const unsigned gy = unsigned(std::max(1, std::min(8, nv / 1024)));
      if ((rc = launch_kernel(xent_grad_f32_kernel, dim3(unsigned(p.T), gy), dim3(256), 0, st, d, ldd, nv,
                              g, status)) != MOE_OK)
        return rc;
      LinearEpi e;
      if (dx) {
        e.out = dx; e.ldo = p.lddx;
        if (!first) { e.res = dx; e.ldr = p.lddx; }
        if ((rc = launch_linear_f32(d, ldd, 1, static_cast<const float*>(W) + v0 * p.ldw, 1, p.ldw, p.T, p.K, nv, e,
                                    r.prod, st)) != MOE_OK)
          return rc;
      }
      if (dW) {
        LinearEpi w;
        w.out = static_cast<float*>(dW) + v0 * p.lddw; w.ldo = p.lddw;
        if ((rc = launch_linear_f32(d, 1, ldd, static_cast<const float*>(x), 1, p.ldx, nv, p.K, p.T, w, r.prod, st)) !=
            MOE_OK)
          return rc;
      }
      continue;
    }
    LinearEpi e;
    e.out = r.d; e.ldo = ldd;
    LinearOperand w = rows_from(b, v0, 2), d{r.d, ldd, false}, xt = a;
    if ((rc = launch_xent_bf16(kXentGrad, a, w, p.T, nv, p.K, e, g, status, st)) != MOE_OK) return rc;
    if (dx) {  // d W: W's rows run along the reduction, so it is read MN-major
      XentEpi s = g;
      LinearEpi o;
      s.ldacc = up8(p.K);
      s.splits = std::min(dx_splits(p), (nv + 63) / 64);
      s.sums = r.split;
      if (!first) s.acc_in = r.acc;
      if (!last) s.acc_out = r.acc;
      else { o.out = dx; o.ldo = p.lddx; }
      w.mn = true;
      if ((rc = launch_xent_bf16(kProductSum, d, w, p.T, p.K, nv, o, s, status, st)) != MOE_OK) return rc;
    }
    if (dW) {  // d^T x: both operands' rows run along the reduction
      LinearEpi o;
      o.out = static_cast<__nv_bfloat16*>(dW) + v0 * p.lddw; o.ldo = p.lddw;
      d.mn = true;
      xt.mn = true;
      if ((rc = launch_xent_bf16(kProductSum, d, xt, nv, p.K, p.T, o, g, status, st)) != MOE_OK) return rc;
    }
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_xent_workspace_bytes(const moe_xent_t* p, int backward, int unaligned, size_t* bytes) {
  moe_xent_t q;
  const int rc = check_xent(p, &q);
  if (rc != MOE_OK) return rc;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = ws_need(q, backward != 0, unaligned != 0);
  return MOE_OK;
}

int moe_xent_forward(const moe_xent_t* p, const void* x, const void* W, const int64_t* target, float* loss, float* lse,
                     float* stats, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_xent_t q;
  const int rc = check_xent(p, &q);
  if (rc != MOE_OK) return rc;
  if (!stats) return MOE_ERR_INVALID_ARG;
  if (q.T == 0) {
    MOE_CUDA_CHECK(cudaMemsetAsync(stats, 0, 8, stream));
    return MOE_OK;
  }
  if (!x || !W || !target || !loss || !lse) return MOE_ERR_INVALID_ARG;
  return forward(q, x, W, target, loss, lse, stats, ws, ws_bytes, stream);
}

int moe_xent_backward(const moe_xent_t* p, const void* x, const void* W, const int64_t* target, const float* lse,
                      const float* dloss, const float* stats, float scale, void* dx, void* dW, void* ws,
                      size_t ws_bytes, moe_stream_t stream) {
  moe_xent_t q;
  const int rc = check_xent(p, &q);
  if (rc != MOE_OK) return rc;
  if (q.T == 0) {
    const size_t eb = q.dtype == MOE_BF16 ? 2 : 4;
    if (dW) MOE_CUDA_CHECK(cudaMemset2DAsync(dW, size_t(q.lddw) * eb, 0, size_t(q.K) * eb, size_t(q.V), stream));
    return MOE_OK;
  }
  if (!x || !W || !target || !lse || (!dloss && !stats)) return MOE_ERR_INVALID_ARG;
  if (!dx && !dW) return MOE_OK;
  return backward(q, x, W, target, lse, dloss, stats, scale, dx, dW, ws, ws_bytes, stream);
}

}  // extern "C"
