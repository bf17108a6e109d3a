// Routing from expert scores with a selection bias, and its gradient.
//
// Lec16 Systems for MoE Models, "DeepSeek V3 MoE": expert groups 8, limited groups 4, top-8 of
// 256; the load balanced by a per-expert bias on the selection. Scores s = sigmoid(l) or
// softmax(l); selection by c = s + b; a group's score the sum of its one or two best c; the
// weights from s alone, renormalised over the choices and scaled.
//
// The choices are those of the scores evaluated in fp64: sigmoid and softmax scores lie close
// together where they saturate, and an order decided in fp32 would depend on the last bits
// of an exponential. Equal fp64 scores rank the lower expert (or group). fp64 runs at 1/64 of
// the fp32 rate, so a token's scores are first formed in fp32 with a bound on their error; only
// when two values that decide (neighbours among the k + 1 best, the last group kept and the
// first one not) lie within that bound is the token taken again in fp64 (choose_fp64). All
// tokens in fp64 took 1640 us for 16384 tokens of 256 experts, top-8 in 4 of 8 groups.
//
// One CTA per chunk of 128 tokens of one group, a warp per token, lane l holding the experts
// l, l + 32, .. (Q = 1, 2, 4 or 8 of them). The CTA then ranks its choices per (choice rank,
// expert) with warp matches and a scan over warps, and writes the chunk's histograms, routed
// counts and loss sums in the form that the scan and finalize kernels of the default routing
// take (route.cu). A batch of one chunk (a serving step) is finished by the same CTA: one
// launch instead of three. Every sum has a fixed order.
#include <algorithm>

#include "route_kernels.cuh"

namespace moe {
namespace {

constexpr int kTokWarps = 16;
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
template <int Q>
__device__ __noinline__ int choose_fp64(const float (&l)[Q], const RouteArgs& a, const ScoreArgs& sc,
                                        double* row) {
  const int lane = threadIdx.x & 31, E = a.E;
  double c[Q];
  if (sc.sigmoid) {
#pragma unroll
    for (int q = 0; q < Q; ++q) c[q] = 1.0 / (1.0 + exp(-double(l[q])));
  } else {
    float mf = -INFINITY;
#pragma unroll
    for (int q = 0; q < Q; ++q) mf = fmaxf(mf, l[q]);
    const double m = double(warp_max(mf));
    double s = 0.0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      c[q] = l[q] > -INFINITY ? exp(double(l[q]) - m) : 0.0;
      s += c[q];
    }
    s = warp_sum(s);
#pragma unroll
    for (int q = 0; q < Q; ++q) c[q] = c[q] / s;
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = lane + 32 * q;
    const float b = sc.bias && e < E ? __ldg(sc.bias + e) : 0.f;
    c[q] = l[q] > -INFINITY && isfinite(b) ? c[q] + double(b) : -INFINITY;
  }
  unsigned groups = kFull;
  if (a.ng > 1) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
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
  for (int q = 0; q < Q; ++q) {
    const int e = lane + 32 * q;
    if (e < E && (a.ng <= 1 || ((groups >> (e / a.gsz)) & 1u))) open |= 1u << q;
  }
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    double bv = -INFINITY;
    int bi = 0x7fffffff;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
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

// Order-preserving map of a float to unsigned and back (finite values).
__device__ __forceinline__ unsigned order_key(float v) {
  const unsigned b = __float_as_uint(v);
  return b ^ (unsigned(int(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(unsigned k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// The loss terms and choice of one token in the general form: any finite logits, -inf where an
// expert is out. q: the normalised scores.
template <int Q>
__device__ __noinline__ int token_general(const float (&l)[Q], const float* lr, const RouteArgs& a,
                                          const ScoreArgs& sc, double* row, float (&q)[Q], float& lse,
                                          float& w) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < Q; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
  const bool any = m > -INFINITY;
  if (!any) m = 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    q[i] = expf(l[i] - m);
    s += q[i];
  }
  s = warp_sum(s);
  lse = any ? m + logf(s) : 0.f;
  const float inv = s > 0.f ? 1.f / s : 0.f;
  float ti = inv;
  if (sc.sigmoid) {
    const float top = fminf(m, 0.f);
    float tot = 0.f;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      q[i] = sigmoid_shifted(l[i], top);
      tot += q[i];
    }
    tot = warp_sum(tot);
    ti = tot > 0.f ? 1.f / tot : 0.f;
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) q[i] *= ti;
  const int id = choose_fp64<Q>(l, a, sc, row);
  float lsel = -INFINITY;
  if (lane < a.k) {
    lsel = __ldg(lr + id);
    if (!isfinite(lsel) || (sc.bias && !isfinite(__ldg(sc.bias + id)))) lsel = -INFINITY;
  }
  w = choice_weight(lsel, lane < a.k, sc, m, inv);
  return id;
}

// The two best keys of every group of 32 m experts (lane-strided experts: slots m g .. of all
// lanes), summed (or the best alone), left in lane g. Equal best keys count twice, as they
// should.
template <int Q>
__device__ __forceinline__ float group_scores_wide(const unsigned (&key)[Q], const RouteArgs& a,
                                                   const ScoreArgs& sc) {
  const int lane = threadIdx.x & 31, per = a.gsz >> 5;
  float gs = -INFINITY;
  for (int g = 0; g < a.ng; ++g) {
    unsigned b1 = 0u, b2 = 0u;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      if (i / per != g) continue;
      const unsigned v = key[i];
      b2 = max(b2, min(b1, v));
      b1 = max(b1, v);
    }
    const unsigned m1 = __reduce_max_sync(kFull, b1);
    float v = order_value(m1 & ~7u);
    if (sc.gtop == 2) {
      const unsigned own = __ballot_sync(kFull, b1 == m1);
      const unsigned second = lane == __ffs(own) - 1 ? b2 : b1;
      v += order_value(__reduce_max_sync(kFull, second) & ~7u);
    }
    if (lane == g) gs = v;
  }
  return gs;
}

// The same for any group size, through this warp's row of shared memory: lane g walks its group
// from a rotated start (the lanes then fall on different banks).
template <int Q>
__device__ __forceinline__ float group_scores_any(const float (&c)[Q], const RouteArgs& a,
                                                  const ScoreArgs& sc, float* row) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < Q; ++i)
    if (lane + 32 * i < a.E) row[lane + 32 * i] = c[i];
  __syncwarp();
  float b1 = -INFINITY, b2 = -INFINITY;
  if (lane < a.ng) {
    int r = lane % a.gsz;
    for (int i = 0; i < a.gsz; ++i) {
      const float v = row[lane * a.gsz + r];
      b2 = fmaxf(b2, fminf(b1, v));
      b1 = fmaxf(b1, v);
      r = r + 1 == a.gsz ? 0 : r + 1;
    }
  }
  __syncwarp();
  return sc.gtop == 2 && a.gsz > 1 ? b1 + b2 : b1;
}

// A token in fp32: false when a decision lies within the error bound (or the values leave the
// range the bound holds for), and the caller takes token_general. With x = __expf(l) (relative
// error (2 + 1.2 |l|) 2^-23), s = sum x in (e^-20, e^20):
//   sigmoid x / (1 + x): |l| sigma (1 - sigma) <= 0.224 and 2 ulp of the division bound the
//     error by 2.5 * 2^-23, and by 27 * 2^-23 of the score where all are small (|l| < 20);
//   softmax x / s: by (13 + 3 * 20) * 2^-23 of the score.
// The bias adds half an ulp, and the keys drop 3 bits for the slot number: at most 2^-20 of the
// largest selection value in all.
template <int Q>
__device__ __forceinline__ bool token_fast(const float (&l)[Q], const float (&b)[Q], float bmax,
                                           const RouteArgs& a, const ScoreArgs& sc, float* row,
                                           float (&q)[Q], float& lse, int& id) {
  const int lane = threadIdx.x & 31;
  constexpr float kU = 1.1920929e-7f;  // 2^-23
  float s = 0.f, tot = 0.f, qm = 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const float x = __expf(l[i]);  // -inf (no expert): 0
    s += x;
    q[i] = sc.sigmoid ? __fdividef(x, 1.f + x) : x;
    tot += q[i];
    qm = fmaxf(qm, q[i]);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    s += __shfl_xor_sync(kFull, s, off);
    tot += __shfl_xor_sync(kFull, tot, off);
  }
  if (!(s > 2.1e-9f && s < 4.8e8f)) return false;
  lse = logf(s);
  const float ti = __fdividef(1.f, tot);
  qm = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(qm)));  // >= 0
  float err;
  if (sc.sigmoid) {
    err = fminf(2.5f, 27.f * qm) * kU;
  } else {
    qm *= ti;
    err = 73.f * qm * kU;
  }
  const float cmax = qm + bmax;
  const float gap = 2.f * err + 1.1f * 8.f * kU * cmax;  // 2^-20 and the rounding of c

  float c[Q];
  unsigned key[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const float sv = sc.sigmoid ? q[i] : q[i] * ti;
    q[i] *= ti;
    c[i] = sv + b[i];
    key[i] = lane + 32 * i < a.E ? ((order_key(c[i]) & ~7u) | unsigned(i)) : 0u;
  }
  if (a.ng > 1) {
    const float gs = (a.gsz & 31) == 0 ? group_scores_wide<Q>(key, a, sc) : group_scores_any<Q>(c, a, sc, row);
    int before = 0;
    for (int h = 0; h < a.ng; ++h) {
      const float vh = __shfl_sync(kFull, gs, h);
      if (vh > gs || (vh == gs && h < lane)) ++before;
    }
    const bool mine = lane < a.ng, kept = mine && before < a.tg;
    if (a.tg < a.ng) {  // the last group kept and the first one not, 2 err each way apart
      const unsigned lo = __reduce_min_sync(kFull, kept ? order_key(gs) : 0xffffffffu);
      const unsigned hi = __reduce_max_sync(kFull, mine && !kept ? order_key(gs) : 0u);
      if (!(order_value(lo) - order_value(hi) > 2.f * gap + 4.f * kU * cmax)) return false;
    }
    const unsigned groups = __ballot_sync(kFull, kept);
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int e = lane + 32 * i;
      const int g = int((unsigned(e) * a.gm24) >> 24);
      if (!((groups >> g) & 1u)) key[i] = 0u;
    }
  }
  unsigned lk = 0u;
#pragma unroll
  for (int i = 0; i < Q; ++i) lk = max(lk, key[i]);
  float prev = INFINITY;
  id = 0;
  for (int j = 0; j <= a.k; ++j) {
    const unsigned top = __reduce_max_sync(kFull, lk);
    if (top == 0u) break;  // j == k: no expert is left
    const unsigned own = __ballot_sync(kFull, lk == top);
    const float v = order_value(top & ~7u);
    if (!(prev - v > gap) || (own & (own - 1u))) return false;
    prev = v;
    if (j == a.k) break;
    const int owner = __ffs(own) - 1;
    if (lane == j) id = owner + 32 * int(top & 7u);
    const bool pop = lane == owner;
    lk = 0u;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      if (pop && key[i] == top) key[i] = 0u;
      lk = max(lk, key[i]);
    }
  }
  return true;
}

template <int Q, bool ONE>
__global__ void __launch_bounds__(kTokThreads, 1) route_scored_kernel(RouteArgs a, ScoreArgs sc) {
  // [warps][E] doubles of group scratch, then [warps][E] probability sums, then the counts
  // [k][4][E]
  extern __shared__ double s_dyn[];
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

  float b[Q];
  float bmax = 0.f;
  bool bias_bad = false;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int e = lane + 32 * i;
    b[i] = sc.bias && e < E ? __ldg(sc.bias + e) : 0.f;
    if (!isfinite(b[i])) bias_bad = true;
    bmax = fmaxf(bmax, fabsf(b[i]));
  }
  bias_bad = __any_sync(kFull, bias_bad);
  bmax = warp_max(bmax);
  if (bias_bad && tid == 0) atomicOr(a.status, kStatusNonfinite);
  double* scratch = s_dyn + size_t(warp) * E;
  float pp[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) pp[i] = 0.f;
  float zacc = 0.f;
  float next[Q];
  auto fetch = [&](int i) {
#pragma unroll
    for (int x = 0; x < Q; ++x) {
      const int e = lane + 32 * x;
      next[x] = (i < nt && e < E) ? __ldg(a.logits + int64_t(t0 + i) * E + e) : -INFINITY;
    }
  };
  fetch(warp);
  for (int i = warp; i < nt; i += kTokWarps) {
    const int64_t t = t0 + i;
    float l[Q], q[Q];
    bool bad = false;
#pragma unroll
    for (int x = 0; x < Q; ++x) {
      l[x] = next[x];
      if (lane + 32 * x < E && !isfinite(l[x])) {
        bad = true;
        l[x] = -INFINITY;
      }
    }
    fetch(i + kTokWarps);  // the warp's next token, while this one is worked on
    bad = __any_sync(kFull, bad);
    float lse, w;
    int id;
    const float* lr = a.logits + t * E;
    bool fast = !bad && !bias_bad &&
                token_fast<Q>(l, b, bmax, a, sc, reinterpret_cast<float*>(scratch), q, lse, id);
    if (fast) {  // the weights, from accurate exponentials of the choices' logits (lanes j < k)
      const float ls = lane < k ? __ldg(lr + id) : 0.f;
      if (sc.renorm) {
        w = lane < k ? (sc.sigmoid ? sigmoid_shifted(ls, 0.f) : expf(ls)) : 0.f;
        float tot = w;
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) tot += __shfl_xor_sync(kFull, tot, off);
        tot = __shfl_sync(kFull, tot, 0);
        fast = tot > 1e-30f;  // else chosen by their biases, with scores that underflow
        w = w / tot;
      } else {
        w = sc.sigmoid ? sigmoid_shifted(ls, 0.f) : expf(ls - lse);
      }
      w *= sc.scale;
    }
    if (!fast) {
      if (bad && lane == 0) atomicOr(a.status, kStatusNonfinite);
      id = token_general<Q>(l, lr, a, sc, scratch, q, lse, w);
    }
#pragma unroll
    for (int x = 0; x < Q; ++x) pp[x] += q[x];
    zacc += lse * lse;
    if (lane < k) {
      a.expert_id[t * k + lane] = id;
      a.gate[t * k + lane] = w;
      s_id[i * kMaxK + lane] = uint8_t(id);
    }
  }
  __syncthreads();  // the group scratch is free
  float* s_pp = reinterpret_cast<float*>(s_dyn);
#pragma unroll
  for (int i = 0; i < Q; ++i)
    if (lane + 32 * i < E) s_pp[warp * E + lane + 32 * i] = pp[i];
  if (lane == 0) s_z[warp] = zacc;
  __syncthreads();
  float psum = 0.f;  // of expert tid
  if (tid < E) {
#pragma unroll
    for (int w = 0; w < kTokWarps; ++w) psum += s_pp[w * E + tid];
    if (!ONE) a.ppart[size_t(c) * E + tid] = psum;
  }
  float sz = 0.f;
  if (tid == 0) {
    for (int w = 0; w < kTokWarps; ++w) sz += s_z[w];
    if (!ONE) a.zpart[c] = sz;
  }
  __syncthreads();

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
  if constexpr (!ONE) {
    for (int x = tid; x < E; x += kTokThreads) {  // choice ranks in order: expert x's columns
      int all = 0;
      for (int j = 0; j < k; ++j) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          int* cw = s_cnt + (j * kWarps + w) * E + x;
          const int v = *cw;
          *cw = run;
          run += v;
        }
        a.hist[(size_t(c) * k + j) * E + x] = run;
        all += run;
      }
      a.hroute[size_t(c) * E + x] = all;  // every choice is a candidate
    }
    __syncthreads();
    for (int x = tid; x < nt * k; x += kTokThreads) {
      const int i = x / k, j = x - i * k;
      const int e = int(s_id[i * kMaxK + j]);
      a.rank[size_t(t0) * k + x] = s_cnt[(j * kWarps + (i >> 5)) * E + e] + int(s_rk[i * kMaxK + j]);
    }
  } else {
    // the whole batch is here: slots, offsets, rows and losses as the scan and finalize
    // kernels form them
    __shared__ int s_first[kMaxE], s_wsum[kMaxE / 32];
    __shared__ float s_aux[kMaxE / 32];
    int all = 0, kept = 0;
    if (tid < E) {
      for (int j = 0; j < k; ++j)
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          int* cw = s_cnt + (j * kWarps + w) * E + tid;
          const int v = *cw;
          *cw = all;
          all += v;
        }
      kept = a.C >= 0 && all > a.C ? a.C : all;
      a.counts[tid] = kept;
      a.counts_routed[tid] = all;
    }
    int inc = kept;
    float aux = tid < E ? float(all) * psum : 0.f;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(kFull, inc, off);
      if (lane >= off) inc += v;
    }
    aux = warp_sum(aux);
    if (warp < kMaxE / 32) {
      if (lane == 31) s_wsum[warp] = inc;
      if (lane == 0) s_aux[warp] = aux;
    }
    __syncthreads();
    if (tid < E) {
      int base = 0;
      for (int w = 0; w < warp; ++w) base += s_wsum[w];
      s_first[tid] = base + inc - kept;
      a.offsets[tid] = base + inc - kept;
      if (tid == E - 1) a.offsets[E] = base + inc;
    }
    if (tid == 0) {
      float t = 0.f;
      for (int w = 0; w < (E + 31) / 32; ++w) t += s_aux[w];
      *a.aux = float(double(t) * (double(E) / (double(a.Sg) * k * double(a.Sg))));
      *a.z = sz / float(a.S);
    }
    __syncthreads();
    for (int x = tid; x < nt * k; x += kTokThreads) {
      const int i = x / k, j = x - i * k;
      const int e = int(s_id[i * kMaxK + j]);
      const int slot = s_cnt[(j * kWarps + (i >> 5)) * E + e] + int(s_rk[i * kMaxK + j]);
      const bool in = a.C < 0 || slot < a.C;
      const int row = in ? s_first[e] + slot : -1;
      const float w = a.gate[x];
      a.pos[x] = in ? slot : -1;
      a.row[x] = row;
      a.drop[x] = in ? MOE_KEPT : MOE_DROP_CAPACITY;
      if (in) {
        a.token_of[row] = i;
        a.w_perm[row] = w;
      } else {
        a.gate[x] = 0.f;
      }
    }
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
  RouteArgs a = route_args(c, C, logits, nullptr, out, ws, L);
  a.gm24 = a.ng > 1 ? ((1u << 24) + unsigned(a.gsz) - 1u) / unsigned(a.gsz) : 0u;
  const size_t dyn = std::max(size_t(kTokWarps) * c.E * sizeof(double), size_t(c.k) * kWarps * c.E * 4);
  const bool one = L.n_chunks == 1 && !d;
  auto go = [&](auto kern) {
    return launch_kernel(kern, dim3(unsigned(L.n_chunks)), dim3(kTokThreads), dyn, st, a,
                         score_args(sc, select_bias));
  };
  int rc;
  if (c.E <= 32) rc = one ? go(route_scored_kernel<1, true>) : go(route_scored_kernel<1, false>);
  else if (c.E <= 64) rc = one ? go(route_scored_kernel<2, true>) : go(route_scored_kernel<2, false>);
  else if (c.E <= 128) rc = one ? go(route_scored_kernel<4, true>) : go(route_scored_kernel<4, false>);
  else rc = one ? go(route_scored_kernel<8, true>) : go(route_scored_kernel<8, false>);
  if (rc != MOE_OK || one) return rc;
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
