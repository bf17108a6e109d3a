// Routing from expert scores with a selection bias, and its gradient.
//
// Lec16 Systems for MoE Models, "DeepSeek V3 MoE": expert groups 8, limited groups 4, top-8 of
// 256; the load balanced by a per-expert bias on the selection. Scores s = sigmoid(l) or
// softmax(l); selection by c = s + b; a group's score the sum of its one or two best c; the
// weights from s alone, renormalised over the choices and scaled.
//
// The choices are those of the scores evaluated in fp64: sigmoid and softmax scores lie close
// together where they saturate, and an order decided in fp32 would depend on the last bits
// of an exponential. Equal fp64 scores rank the lower expert (or group).
//
// One CTA per chunk of 128 tokens of one group, a warp per token, lane l holding the experts
// l, l + 32, .. (at most 8). The CTA then ranks its choices per (choice rank, expert) with warp
// matches and a scan over warps, and writes the chunk's histograms, routed counts and loss
// sums in the form that the scan and finalize kernels of the default routing take
// (route.cu). Every sum has a fixed order.
#include <algorithm>

#include "route_kernels.cuh"

namespace moe {
namespace {

constexpr int kTokWarps = 8;
constexpr int kTokThreads = 32 * kTokWarps;
constexpr unsigned kFull = 0xffffffffu;

struct ScoreArgs {
  const float* bias;  // select_bias, nullable
  int sigmoid, gtop, renorm;
  float scale;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
  return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

// exp(min(l, 0) - m) / (1 + exp(-|l|)) = sigmoid(l) exp(-m): with m = 0 the sigmoid itself
// (no overflow for any l), with m the largest min(l, 0) of a set the terms of its
// renormalised sigmoids, which then cannot all underflow. l = -inf gives 0.
__device__ __forceinline__ float sigmoid_shifted(float l, float m) {
  return l > -INFINITY ? expf(fminf(l, 0.f) - m) / (1.f + expf(-fabsf(l))) : 0.f;
}

// A token's choices by the fp64 scores: lane j < k gets the j-th one's index. l: the lane's
// logits (-inf where the expert is out), own: its experts that exist, row: E doubles of this
// warp in shared memory.
__device__ __noinline__ int choose_fp64(const float (&l)[8], const RouteArgs& a, const ScoreArgs& sc,
                                        double* row) {
  const int lane = threadIdx.x & 31, E = a.E;
  double c[8];
  if (sc.sigmoid) {
#pragma unroll
    for (int q = 0; q < 8; ++q) c[q] = 1.0 / (1.0 + exp(-double(l[q])));
  } else {
    float mf = -INFINITY;
#pragma unroll
    for (int q = 0; q < 8; ++q) mf = fmaxf(mf, l[q]);
    const double m = double(warp_max(mf));
    double s = 0.0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      c[q] = l[q] > -INFINITY ? exp(double(l[q]) - m) : 0.0;
      s += c[q];
    }
    s = warp_sum(s);
#pragma unroll
    for (int q = 0; q < 8; ++q) c[q] = c[q] / s;
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int e = lane + 32 * q;
    const float b = sc.bias && e < E ? __ldg(sc.bias + e) : 0.f;
    c[q] = l[q] > -INFINITY && isfinite(b) ? c[q] + double(b) : -INFINITY;
  }
  unsigned groups = kFull;
  if (a.ng > 1) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (lane + 32 * q < E) row[lane + 32 * q] = c[q];
    __syncwarp();
    double gs = -INFINITY;
    if (lane < a.ng) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < a.gsz; ++i) {
        const double v = row[lane * a.gsz + i];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
      gs = (sc.gtop == 2 && a.gsz > 1) ? b1 + b2 : b1;
    }
    int before = 0;
    for (int h = 0; h < a.ng; ++h) {
      const double vh = __shfl_sync(kFull, gs, h);
      if (vh > gs || (vh == gs && h < lane)) ++before;
    }
    groups = __ballot_sync(kFull, lane < a.ng && before < a.tg);
    __syncwarp();
  }
  unsigned open = 0u;  // bit q: expert lane + 32 q may still be chosen
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int e = lane + 32 * q;
    if (e < E && (a.ng <= 1 || ((groups >> (e / a.gsz)) & 1u))) open |= 1u << q;
  }
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    double bv = -INFINITY;
    int bi = 0x7fffffff;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int e = lane + 32 * q;
      if (((open >> q) & 1u) && (c[q] > bv || (c[q] == bv && e < bi))) {
        bv = c[q];
        bi = e;
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const double ov = __shfl_xor_sync(kFull, bv, off);
      const int oi = __shfl_xor_sync(kFull, bi, off);
      if (ov > bv || (ov == bv && oi < bi)) {
        bv = ov;
        bi = oi;
      }
    }
    if ((bi & 31) == lane) open &= ~(1u << (bi >> 5));
    if (lane == j) mine = bi;
  }
  return mine;
}

// The weight of this lane's choice (lanes j < k; lsel its logit, -inf when it is out), from
// the scores of the k choices; m, inv: the token's largest logit and 1 / sum exp(l - m)
// (softmax).
__device__ __forceinline__ float choice_weight(float lsel, bool on, const ScoreArgs& sc, float m,
                                               float inv) {
  if (!on) lsel = -INFINITY;
  float w;
  if (sc.renorm) {
    float top = warp_max(sc.sigmoid ? fminf(lsel, 0.f) : lsel);
    if (!(top > -INFINITY)) top = 0.f;
    w = sc.sigmoid ? sigmoid_shifted(lsel, top) : (lsel > -INFINITY ? expf(lsel - top) : 0.f);
    const float tot = warp_sum(w);
    w = tot > 0.f ? w / tot : 0.f;
  } else {
    w = sc.sigmoid ? sigmoid_shifted(lsel, 0.f) : (lsel > -INFINITY ? expf(lsel - m) * inv : 0.f);
  }
  return w * sc.scale;
}

__global__ void __launch_bounds__(kTokThreads) route_scored_kernel(RouteArgs a, ScoreArgs sc) {
  extern __shared__ double s_dyn[];  // [8 warps][E] group scratch, then the counts [k][4][E]
  __shared__ float s_pp[kTokWarps][kMaxE];
  __shared__ float s_z[kTokWarps];
  __shared__ uint8_t s_id[kThreads * kMaxK];
  __shared__ uint8_t s_rk[kThreads * kMaxK];
  const int c = blockIdx.x;
  const int g = c / a.n_cpg, cc = c % a.n_cpg;
  const int t0 = g * a.Sg + cc * kThreads;
  const int nt = min(kThreads, a.Sg - cc * kThreads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = a.E, k = a.k;
  pdl_wait();
  pdl_trigger();
  if (c == 0 && tid == 0) *a.done = 0u;  // ticket counter of route_scan_kernel

  if (sc.bias && tid < E && !isfinite(__ldg(sc.bias + tid))) atomicOr(a.status, kStatusNonfinite);
  float pp[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float zacc = 0.f;
  for (int i = warp; i < nt; i += kTokWarps) {
    const int64_t t = t0 + i;
    const float* lr = a.logits + t * E;
    float l[8];
    bool bad = false;
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int e = lane + 32 * q;
      l[q] = -INFINITY;
      if (e < E) {
        const float v = __ldg(lr + e);
        if (isfinite(v)) l[q] = v;
        else bad = true;
      }
      m = fmaxf(m, l[q]);
    }
    if (bad) atomicOr(a.status, kStatusNonfinite);
    m = warp_max(m);
    const bool any = m > -INFINITY;
    if (!any) m = 0.f;
    // logsumexp, and the normalised scores for the balance loss
    float x[8], s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      x[q] = expf(l[q] - m);
      s += x[q];
    }
    s = warp_sum(s);
    const float lse = any ? m + logf(s) : 0.f;
    const float inv = s > 0.f ? 1.f / s : 0.f;
    if (sc.sigmoid) {
      const float top = fminf(m, 0.f);
      float tot = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        x[q] = sigmoid_shifted(l[q], top);
        tot += x[q];
      }
      tot = warp_sum(tot);
      const float ti = tot > 0.f ? 1.f / tot : 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) pp[q] += x[q] * ti;
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) pp[q] += x[q] * inv;
    }
    zacc += lse * lse;
    const int id = choose_fp64(l, a, sc, s_dyn + size_t(warp) * E);
    // lane j's logit of choice j
    float lsel = -INFINITY;
    if (lane < k) {
      lsel = __ldg(lr + id);
      if (!isfinite(lsel) || (sc.bias && !isfinite(__ldg(sc.bias + id)))) lsel = -INFINITY;
    }
    const float w = choice_weight(lsel, lane < k, sc, m, inv);
    if (lane < k) {
      a.expert_id[t * k + lane] = id;
      a.gate[t * k + lane] = w;
      s_id[i * kMaxK + lane] = uint8_t(id);
    }
  }
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (lane + 32 * q < E) s_pp[warp][lane + 32 * q] = pp[q];
  if (lane == 0) s_z[warp] = zacc;
  __syncthreads();
  for (int e = tid; e < E; e += kTokThreads) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kTokWarps; ++w) sum += s_pp[w][e];
    a.ppart[size_t(c) * E + e] = sum;
  }
  if (tid == 0) {
    float sz = 0.f;
    for (int w = 0; w < kTokWarps; ++w) sz += s_z[w];
    a.zpart[c] = sz;
  }

  // rank of each choice among the chunk's earlier ones of the same (j, e): the first
  // kThreads threads hold a token each; counts per (j, warp, e), one scan over the warps
  int* s_cnt = reinterpret_cast<int*>(s_dyn);
  for (int x = tid; x < k * kWarps * E; x += kTokThreads) s_cnt[x] = 0;
  __syncthreads();
  const unsigned lt_mask = (1u << lane) - 1u;
  if (tid < kThreads) {
    for (int j = 0; j < k; ++j) {
      const bool on = tid < nt;
      const int e = on ? int(s_id[tid * kMaxK + j]) : -1;
      const unsigned peers = __match_any_sync(kFull, on ? e : 1024 + lane);
      const int rk = __popc(peers & lt_mask);
      s_rk[tid * kMaxK + j] = uint8_t(rk);
      if (on && rk == 0) s_cnt[(j * kWarps + warp) * E + e] = __popc(peers);
    }
  }
  __syncthreads();
  for (int x = tid; x < k * E; x += kTokThreads) {
    const int j = x / E, e = x - j * E;
    int run = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      int* cw = s_cnt + (j * kWarps + w) * E + e;
      const int v = *cw;
      *cw = run;
      run += v;
    }
    a.hist[(size_t(c) * k + j) * E + e] = run;
  }
  __syncthreads();
  if (tid < nt) {
    for (int j = 0; j < k; ++j) {
      const int e = int(s_id[tid * kMaxK + j]);
      a.rank[size_t(t0 + tid) * k + j] = s_cnt[(j * kWarps + warp) * E + e] + int(s_rk[tid * kMaxK + j]);
    }
  }
  for (int e = tid; e < E; e += kTokThreads) {
    int run = 0;  // every choice is a candidate: the routed counts are the histograms' sums
    for (int j = 0; j < k; ++j) run += a.hist[(size_t(c) * k + j) * E + e];
    a.hroute[size_t(c) * E + e] = run;
  }
}

// dlogits of one token per warp. With q_e the normalised scores (softmax: the probabilities
// p_e), f the routed fractions of the token's group, w^_j the choices' renormalised scores
// and d_j their gradients (0 where not kept):
//   sigmoid   renorm:  dl_j  = scale w^_j (1 - s_j) (d_j - sum_i d_i w^_i)
//             else:    dl_j  = scale d_j s_j (1 - s_j)
//             aux:     dl_e += ca q_e (1 - s_e) (f_e - sum f q)
//   softmax   renorm:  dl_j  = scale w^_j (d_j - sum_i d_i w^_i)
//             else:    dl_j  = scale p_j d_j, dl_e -= scale p_e sum_i d_i p_i
//             aux:     dl_e += ca p_e (f_e - sum f p)
//   z         dl_e += 2 cz / S lse p_e
// with ca = aux_coef E / (G S_g). 1 - s is evaluated as sigmoid(-l), so it keeps its precision
// where s is close to 1.
__global__ void __launch_bounds__(256)
    route_scored_bwd_kernel(const float* __restrict__ logits, const int32_t* __restrict__ expert_id,
                            const int32_t* __restrict__ row, const int32_t* __restrict__ counts_routed,
                            const float* __restrict__ dgate, const float* __restrict__ gpart,
                            int n_tiles, int S, int G, int E, int k, ScoreArgs sc, float aux_coef,
                            float z_coef, float* __restrict__ dlogits,
                            __nv_bfloat16* __restrict__ dlb, int Ep) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (t >= S) return;
  const float* lr = logits + t * E;
  float l[8], p[8], dl[8];
  float m = -INFINITY;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int e = lane + 32 * q;
    l[q] = e < E ? __ldg(lr + e) : -INFINITY;
    if (!isfinite(l[q])) l[q] = -INFINITY;
    m = fmaxf(m, l[q]);
    dl[q] = 0.f;
  }
  m = warp_max(m);
  const bool any = m > -INFINITY;
  if (!any) m = 0.f;
  float s = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    p[q] = expf(l[q] - m);
    s += p[q];
  }
  s = warp_sum(s);
  const float inv = s > 0.f ? 1.f / s : 0.f, lse = any ? m + logf(s) : 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) p[q] *= inv;

  // the choices, lane j < k: expert, logit, gradient of its weight
  int id = -1;
  float lsel = -INFINITY, dg = 0.f;
  if (lane < k) {
    id = expert_id[t * k + lane];
    if (id < 0 || id >= E) id = -1;
    if (id >= 0) lsel = __ldg(lr + id);
    if (!isfinite(lsel)) lsel = -INFINITY;
    const int r = row[t * k + lane];
    if (r >= 0) {
      if (dgate) dg = dgate[t * k + lane];
      else
        for (int nt = 0; nt < n_tiles; ++nt) dg += gpart[int64_t(r) * n_tiles + nt];
    }
  }
  ScoreArgs unit = sc;
  unit.scale = 1.f;
  const float w = choice_weight(lsel, lane < k, unit, m, inv);
  const float inner = (sc.renorm || !sc.sigmoid) ? warp_sum(w * dg) : 0.f;
  float dsel = sc.scale * w * ((sc.renorm ? dg - inner : dg) *
                               (sc.sigmoid ? sigmoid_shifted(-lsel, 0.f) : 1.f));
  if (!(lsel > -INFINITY)) dsel = 0.f;
  for (int j = 0; j < k; ++j) {
    const int idj = __shfl_sync(kFull, id, j);
    const float dj = __shfl_sync(kFull, dsel, j);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (idj == lane + 32 * q) dl[q] += dj;
  }
  if (!sc.sigmoid && !sc.renorm) {
    const float ci = sc.scale * inner;
#pragma unroll
    for (int q = 0; q < 8; ++q) dl[q] -= p[q] * ci;
  }
  if (aux_coef != 0.f) {
    const int Sg = S / G;
    const int32_t* cr = counts_routed + (t / Sg) * E;
    const float fs = 1.f / (float(Sg) * float(k));
    const float ca = aux_coef * float(E) / (float(G) * float(Sg));
    float f[8], x[8], fq = 0.f, ti = 1.f;
    if (sc.sigmoid) {
      const float top = fminf(m, 0.f);
      float tot = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        x[q] = sigmoid_shifted(l[q], top);
        tot += x[q];
      }
      tot = warp_sum(tot);
      ti = tot > 0.f ? 1.f / tot : 0.f;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int e = lane + 32 * q;
      x[q] = sc.sigmoid ? x[q] * ti : p[q];
      f[q] = e < E ? float(cr[e]) * fs : 0.f;
      fq += f[q] * x[q];
    }
    fq = warp_sum(fq);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float one_s = sc.sigmoid && l[q] > -INFINITY ? sigmoid_shifted(-l[q], 0.f) : 1.f;
      dl[q] += ca * x[q] * one_s * (f[q] - fq);
    }
  }
  if (z_coef != 0.f) {
    const float cz = z_coef * 2.f / float(S) * lse;
#pragma unroll
    for (int q = 0; q < 8; ++q) dl[q] += cz * p[q];
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int e = lane + 32 * q;
    if (e < E) dlogits[t * E + e] = dl[q];
    if (dlb && e < Ep) dlb[t * Ep + e] = __float2bfloat16_rn(e < E ? dl[q] : 0.f);
  }
}

ScoreArgs score_args(const moe_score_t& sc, const float* bias) {
  return ScoreArgs{bias, int(sc.score == MOE_SCORE_SIGMOID), sc.group_top, sc.renorm, sc.scale};
}

}  // namespace

int launch_route_scored(const moe_config_t& c, const moe_score_t& sc, int C, const float* logits,
                        const float* select_bias, const moe_route_out_t& out, char* ws,
                        const WsLayout& L, cudaStream_t st, const DispatchFuse* d) {
  const RouteArgs a = route_args(c, C, logits, nullptr, out, ws, L);
  const size_t dyn = std::max(size_t(kTokWarps) * c.E * sizeof(double), size_t(c.k) * kWarps * c.E * 4);
  const int rc = launch_kernel(route_scored_kernel, dim3(unsigned(L.n_chunks)), dim3(kTokThreads), dyn,
                               st, a, score_args(sc, select_bias));
  if (rc != MOE_OK) return rc;
  return launch_scan_finalize(c, a, d, st);
}

int launch_route_scored_backward(const moe_config_t& c, const moe_score_t& sc, const float* logits,
                                 const moe_route_out_t& r, const float* dgate, const float* gpart,
                                 int n_tiles, float aux_coef, float z_coef, float* dlogits, void* dlb,
                                 int Ep, cudaStream_t st) {
  const unsigned blocks = unsigned((int64_t(c.S) * 32 + 255) / 256);
  return launch_kernel(route_scored_bwd_kernel, dim3(blocks), dim3(256), 0, st, logits,
                       static_cast<const int32_t*>(r.expert_id), static_cast<const int32_t*>(r.row),
                       static_cast<const int32_t*>(r.counts_routed), dgate, gpart, n_tiles, c.S, c.G,
                       c.E, c.k, score_args(sc, nullptr), aux_coef, z_coef, dlogits,
                       static_cast<__nv_bfloat16*>(dlb), Ep);
}

}  // namespace moe
