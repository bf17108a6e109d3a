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
// first one not) lie within that bound are those evaluated in fp64, a lane each. All tokens in
// fp64 took 1640 us for 16384 tokens of 256 experts, top-8 in 4 of 8 groups; now 45 us, of
// which this kernel takes 27. It waits on latency: four warps a scheduler (128 CTAs of 16 on 152
// SMs) take 45 % of the issue slots, each warp's 860 instructions a token (an exponential and a
// reciprocal an expert, two warp maxima a group, one a choice) hang together, and a token's logits
// are asked for when its turn comes; issue alone would take 13 us, memory (16.8 MB of logits) 3. 65536
// tokens of 64 experts, top-2, softmax scores, capacity: 39 us, 22 here (52 % of the slots, 1.7 waves
// of CTAs). One token: 10 us alone in a chain of launches.
//
// One CTA per chunk of 128 tokens of one group, a warp per token, lane l holding the experts
// l, l + 32, .. (Q = 1, 2, 4 or 8 of them). The CTA then ranks its choices per (choice rank,
// expert) with warp matches and a scan over warps, and writes the chunk's histograms, routed
// counts and loss sums in the form that the scan and finalize kernels of the default routing
// take (route.cu). A batch of one chunk (a serving step) is finished by the same CTA: one
// launch instead of three. Every sum has a fixed order.
#include <algorithm>
#include <type_traits>

#include "elem.cuh"
#include "route_kernels.cuh"

namespace moe {
namespace {

// The chunk kernel: 16 warps; two CTAs an SM with at most 2 experts a lane (64 registers a
// thread), so that one's last steps run beside the other's tokens. 32 warps with 8 experts a lane
// (64 registers, spills) took the same time.
constexpr int kTokWarps = 16, kTokThreads = 32 * kTokWarps;
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

// Order-preserving map of a double to unsigned (integer comparisons; fp64 ones run on the slow
// pipe): larger value, larger key; -inf is not 0. Back: order_double.
__device__ __forceinline__ unsigned long long order_key(double v) {
  const long long b = __double_as_longlong(v + 0.0);  // -0 and 0 are equal
  return static_cast<unsigned long long>(b) ^ (static_cast<unsigned long long>(b >> 63) | (1ull << 63));
}
__device__ __forceinline__ double order_double(unsigned long long k) {
  return __longlong_as_double(static_cast<long long>(k ^ ((k >> 63) ? (1ull << 63) : ~0ull)));
}

// The token's fp64 sum of exp(l - m) over all experts, m its largest logit (softmax scores).
template <int Q>
__device__ __forceinline__ double softmax_sum(const float (&l)[Q], double m) {
  double s = 0.0;
#pragma unroll
  for (int q = 0; q < Q; ++q) s += l[q] > -INFINITY ? exp(double(l[q]) - m) : 0.0;  // -inf: out
  return warp_sum(s);
}

// A token's choices by the fp64 scores: lane j < k gets the j-th one's index. l: the lane's
// logits (-inf where the expert is out), row: E doubles of this warp in shared memory.
template <int Q>
__device__ __noinline__ int choose_fp64(const float (&l)[Q], const RouteArgs& a, const ScoreArgs& sc,
                                        double* row) {
  const int lane = threadIdx.x & 31, E = a.E;
  double m = 0.0, z = 1.0;
  if (!sc.sigmoid) {
    float mf = -INFINITY;
#pragma unroll
    for (int q = 0; q < Q; ++q) mf = fmaxf(mf, l[q]);
    m = double(warp_max(mf));
    z = softmax_sum<Q>(l, m);
  }
  unsigned long long key[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int e = lane + 32 * q;
    double c = sc.sigmoid ? 1.0 / (1.0 + exp(-double(l[q]))) : exp(double(l[q]) - m) / z;
    const float b = sc.bias && e < E ? __ldg(sc.bias + e) : 0.f;
    c = l[q] > -INFINITY && isfinite(b) ? c + double(b) : -INFINITY;
    key[q] = order_key(c);
  }
  unsigned groups = kFull;
  if (a.ng > 1) {
    unsigned long long* keys = reinterpret_cast<unsigned long long*>(row);
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (lane + 32 * q < E) keys[lane + 32 * q] = key[q];
    __syncwarp();
    unsigned long long gs = 0;
    if (lane < a.ng) {
      unsigned long long b1 = 0, b2 = 0;
      for (int i = 0; i < a.gsz; ++i) {
        const unsigned long long v = keys[lane * a.gsz + i];
        b2 = max(b2, min(b1, v));
        b1 = max(b1, v);
      }
      gs = (sc.gtop == 2 && a.gsz > 1) ? order_key(order_double(b1) + order_double(b2)) : b1;
    }
    int before = 0;
    for (int h = 0; h < a.ng; ++h) {
      const unsigned long long vh = __shfl_sync(kFull, gs, h);
      if (vh > gs || (vh == gs && h < lane)) ++before;
    }
    groups = __ballot_sync(kFull, lane < a.ng && before < a.tg);
    __syncwarp();
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {  // 0: not to be chosen
    const int e = lane + 32 * q;
    if (e >= E || (a.ng > 1 && !((groups >> (e / a.gsz)) & 1u))) key[q] = 0;
  }
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    unsigned long long best = 0;
    int e = 0x7fffffff;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (key[q] > best) {  // equal keys: the lower q first
        best = key[q];
        e = lane + 32 * q;
      }
    const unsigned hi = __reduce_max_sync(kFull, unsigned(best >> 32));
    const bool top = unsigned(best >> 32) == hi;
    const unsigned lo = __reduce_max_sync(kFull, top ? unsigned(best) : 0u);
    const int id = __reduce_min_sync(kFull, top && unsigned(best) == lo ? e : 0x7fffffff);
    if (lane == j) mine = id;
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (lane + 32 * q == id) key[q] = 0;
  }
  return mine;
}

// The loss terms and choice of one token in the general form: any finite logits, -inf where an
// expert is out. q: the normalised scores; the logits' largest m and s = sum exp(l - m) (0 and 0
// where no expert is in). Lane j < k returns choice j.
template <int Q>
__device__ __noinline__ int token_general(const float (&l)[Q], const RouteArgs& a, const ScoreArgs& sc,
                                          double* row, float (&q)[Q], float& m, float& s) {
  m = -INFINITY;
#pragma unroll
  for (int i = 0; i < Q; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
  if (!(m > -INFINITY)) m = 0.f;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    q[i] = expf(l[i] - m);
    s += q[i];
  }
  s = warp_sum(s);
  float ti = s > 0.f ? 1.f / s : 0.f;
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
  return choose_fp64<Q>(l, a, sc, row);
}


// Group scores from keys (bits of non-negative floats, low 3 bits the slot number), lane g
// getting group g's; groups of 32 m experts, i.e. slots m g .. m g + m - 1 of every lane. Equal
// best keys count twice, as they should.
template <int Q>
__device__ __forceinline__ float group_scores_wide(const unsigned (&key)[Q], const RouteArgs& a,
                                                   const ScoreArgs& sc) {
  const int lane = threadIdx.x & 31, per = a.gsz >> 5;
  unsigned b1 = 0u, b2 = 0u, g1 = 0u, g2 = 0u;
  int g = 0, have = 0;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const unsigned v = key[i];
    b2 = max(b2, min(b1, v));
    b1 = max(b1, v);
    if (++have == per) {  // slots g per .. g per + per - 1 are in
      const unsigned m1 = __reduce_max_sync(kFull, b1);
      unsigned m2 = 0u;
      if (sc.gtop == 2) {
        const int owner = __ffs(__ballot_sync(kFull, b1 == m1)) - 1;
        m2 = __reduce_max_sync(kFull, lane == owner ? b2 : b1);
      }
      if (lane == g) {
        g1 = m1;
        g2 = m2;
      }
      ++g;
      have = 0;
      b1 = b2 = 0u;
    }
  }
  return __uint_as_float(g1 & ~7u) + __uint_as_float(g2 & ~7u);
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
  float b1 = 0.f, b2 = 0.f;
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

// Groups of 32, the lanes' slot g being group g.
template <int Q>
__device__ __forceinline__ float group_scores_32(const unsigned (&key)[Q], const ScoreArgs& sc) {
  const int lane = threadIdx.x & 31;
  unsigned g1 = 0u, g2 = 0u;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const unsigned m1 = __reduce_max_sync(kFull, key[i]);
    unsigned m2 = 0u;
    if (sc.gtop == 2) {
      const bool at = key[i] == m1;
      const unsigned own = __ballot_sync(kFull, at);
      m2 = __reduce_max_sync(kFull, at ? 0u : key[i]);
      if (own & (own - 1u)) m2 = m1;  // two experts share the best key
    }
    if (lane == i) {
      g1 = m1;
      g2 = m2;
    }
  }
  return __uint_as_float(g1 & ~7u) + __uint_as_float(g2 & ~7u);
}

// Group g's score by the fp64 sigmoids, as an ordered key; the group's experts a lane each (or
// every 32nd), their logits read again.
__device__ __noinline__ unsigned long long group_score_fp64(const float* lr, const float* bias, int g,
                                                            int gsz, int gtop) {
  const int lane = threadIdx.x & 31;
  unsigned long long b1 = 0, b2 = 0;
  for (int i = lane; i < gsz; i += 32) {
    const int e = g * gsz + i;
    const unsigned long long v =
        order_key(1.0 / (1.0 + exp(-double(__ldg(lr + e)))) + (bias ? double(__ldg(bias + e)) : 0.0));
    b2 = max(b2, min(b1, v));
    b1 = max(b1, v);
  }
  auto top = [&](unsigned long long v) {
    const unsigned hi = __reduce_max_sync(kFull, unsigned(v >> 32));
    const unsigned lo = __reduce_max_sync(kFull, unsigned(v >> 32) == hi ? unsigned(v) : 0u);
    return (static_cast<unsigned long long>(hi) << 32) | lo;
  };
  const unsigned long long m1 = top(b1);
  if (gtop != 2 || gsz == 1) return m1;
  const int owner = __ffs(__ballot_sync(kFull, b1 == m1)) - 1;
  return order_key(order_double(m1) + order_double(top(lane == owner ? b2 : b1)));
}

// How many groups rank before this lane's (lane g < ng holds group g's score).
__device__ __forceinline__ int groups_before(float gs, int ng) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  if (ng <= 8) {  // lane (g, h): group g = lane & 7 against h = lane / 8 and h + 4
    const int g = lane & 7, h = lane >> 3;
    const float vg = __shfl_sync(kFull, gs, g);
    const float v0 = __shfl_sync(kFull, gs, h), v1 = __shfl_sync(kFull, gs, h + 4);
    if (h < ng && (v0 > vg || (v0 == vg && h < g))) ++before;
    if (h + 4 < ng && (v1 > vg || (v1 == vg && h + 4 < g))) ++before;
    before += __shfl_xor_sync(kFull, before, 8);
    before += __shfl_xor_sync(kFull, before, 16);
    return before;
  }
  for (int h = 0; h < ng; ++h) {
    const float vh = __shfl_sync(kFull, gs, h);
    if (vh > gs || (vh == gs && h < lane)) ++before;
  }
  return before;
}

// Of n candidates, a lane each (l its logit, b its bias, id its index): how many rank before this
// lane's by sigmoid(l) + b in fp64, equal ones by index.
__device__ __noinline__ int rank_fp64(float l, float b, int id, int n) {
  const unsigned long long key = order_key(1.0 / (1.0 + exp(-double(l))) + double(b));
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const unsigned long long o = __shfl_sync(kFull, key, i);
    const int oid = __shfl_sync(kFull, id, i);
    if (o > key || (o == key && oid < id)) ++rank;
  }
  return rank;
}

// A token in fp32. Sigmoid scores that decide and lie within the error bound of each other (the
// groups at the border of the kept ones, neighbours among the choices) are evaluated in fp64, a
// lane each. False where softmax scores, whose sum all experts enter, lie that close, or the
// values leave the range the bound holds for: the caller then takes token_general.
// l: the lane's finite logits (-1e30 where there is no expert), b: the biases less the smallest
// one, so that every selection value c = s + b is >= 0 and its bits order as an integer. The low
// 3 bits of a key give way to the lane's slot number, so one warp maximum finds the value and
// its expert; a key below 8 is no expert.
// With x = exp2(l log2 e) (relative error (2 + 1.2 |l|) 2^-23), s = sum x in (e^-20, e^20):
//   sigmoid x / (1 + x): |l| sigma (1 - sigma) <= 0.224 and 2 ulp of the reciprocal bound the
//     error by 2.5 * 2^-23, and by 27 * 2^-23 of the score where all are small (|l| < 20);
//   softmax x / s: by (13 + 3 * 20) * 2^-23 of the score.
// The shifted bias and the sum c add an ulp (2^-23 of the largest value), the dropped bits 7.
// Writes the choices to ids, and s.
template <int Q, bool SIG>
__device__ __forceinline__ bool token_fast(const float (&l)[Q], const float (&b)[Q], float brange,
                                           const float* lr, const RouteArgs& a, const ScoreArgs& sc,
                                           float* row, float (&pp)[Q], uint8_t* ids, float& s_out) {
  const int lane = threadIdx.x & 31;
  constexpr float kU = 1.1920929e-7f;  // 2^-23
  float q[Q];
  float s = 0.f, tot = 0.f, wild = 0.f;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const float x = exp2_approx(l[i] * 1.44269504088896341f);
    wild = fmaf(l[i], 0.f, wild);  // NaN when a logit is not finite
    s += x;
    if constexpr (SIG) {
      q[i] = x * rcp_approx(1.f + x);
      tot += q[i];
    } else {
      q[i] = x;
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    s += __shfl_xor_sync(kFull, s, off);
    if constexpr (SIG) tot += __shfl_xor_sync(kFull, tot, off);
  }
  if (__any_sync(kFull, !(wild == 0.f)) || !(s > 2.1e-9f && s < 4.8e8f)) return false;
  s_out = s;
  const float ti = rcp_approx(SIG ? tot : s);
  float err, qm;  // qm: at least the largest score
  if constexpr (SIG) {
    qm = fminf(tot, 1.f);
    err = fminf(2.5f, 27.f * qm) * kU;
  } else {
    qm = q[0];
#pragma unroll
    for (int i = 1; i < Q; ++i) qm = fmaxf(qm, q[i]);
    qm = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(qm))) * ti;
    err = 73.f * qm * kU;
  }
  const float cmax = qm + brange;
  const float gap = 2.f * err + 10.f * kU * cmax;

  float c[Q];
  unsigned key[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    c[i] = SIG ? q[i] + b[i] : fmaf(q[i], ti, b[i]);
    key[i] = (__float_as_uint(c[i]) & ~7u) | unsigned(i);
  }
  if (a.ng > 1) {
    const float gs = a.gsz == 32          ? group_scores_32<Q>(key, sc)
                     : (a.gsz & 31) == 0 ? group_scores_wide<Q>(key, a, sc)
                                         : group_scores_any<Q>(c, a, sc, row);
    const int before = groups_before(gs, a.ng);  // every lane: it shuffles
    const bool mine = lane < a.ng;
    bool kept = mine && before < a.tg;
    if (a.tg < a.ng) {  // the last group kept and the first one not
      const float lo = __uint_as_float(__reduce_min_sync(kFull, kept ? __float_as_uint(gs) : 0x7f800000u));
      const float hi = __uint_as_float(__reduce_max_sync(kFull, mine && !kept ? __float_as_uint(gs) : 0u));
      const float margin = 2.f * gap + 4.f * kU * cmax;
      if (!(lo - hi > margin)) {
        if constexpr (!SIG) return false;
        // the groups within the bound of the border: the best of them by their fp64 scores
        const bool near = mine && (kept ? !(gs - hi > margin) : !(lo - gs > margin));
        const unsigned close = __ballot_sync(kFull, near);
        const int seats = a.tg - __popc(__ballot_sync(kFull, kept && !near));
        unsigned long long score = 0;
        for (unsigned todo = close; todo; todo &= todo - 1u) {
          const int g = __ffs(todo) - 1;
          const unsigned long long v = group_score_fp64(lr, sc.bias, g, a.gsz, sc.gtop);
          if (lane == g) score = v;
        }
        int rank = 0;
        for (unsigned todo = close; todo; todo &= todo - 1u) {
          const int g = __ffs(todo) - 1;
          const unsigned long long o = __shfl_sync(kFull, score, g);
          if (o > score || (o == score && g < lane)) ++rank;
        }
        if (near) kept = rank < seats;
      }
    }
    const unsigned groups = __ballot_sync(kFull, kept);
    if (a.gsz == 32) {
#pragma unroll
      for (int i = 0; i < Q; ++i) key[i] = (groups >> i) & 1u ? key[i] : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int g = int((unsigned(lane + 32 * i) * a.gm24) >> 24);
        if (!((groups >> g) & 1u)) key[i] = 0u;
      }
    }
  }
  // each lane's keys in falling order (odd-even transposition), so that taking one shifts them
#pragma unroll
  for (int r = 0; r < Q; ++r)
#pragma unroll
    for (int i = r & 1; i + 1 < Q; i += 2) {
      const unsigned hi = max(key[i], key[i + 1]);
      key[i + 1] = min(key[i], key[i + 1]);
      key[i] = hi;
    }
  unsigned mine = 0u;  // lane j: the j-th largest key, and its lane
  int from = 0;
  auto take = [&](int j, unsigned top) {
    const int owner = __ffs(__ballot_sync(kFull, key[0] == top)) - 1;
    if (lane == j) {
      mine = top;
      from = owner;
    }
    const bool pop = lane == owner;
#pragma unroll
    for (int i = 0; i < Q; ++i) key[i] = pop ? (i + 1 < Q ? key[i + 1 < Q ? i + 1 : 0] : 0u) : key[i];
  };
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    if (j == a.k) break;
    take(j, __reduce_max_sync(kFull, key[0]));
  }
  unsigned last = __reduce_max_sync(kFull, key[0]);  // the best one not chosen
  const float v = __uint_as_float((lane == a.k ? last : mine) & ~7u);
  const float above = __shfl_up_sync(kFull, v, 1);
  const bool close = lane > 0 && (lane < a.k || (lane == a.k && last >= 8u)) && !(above - v > gap);
  int id = from + 32 * int(mine & 7u);
  if (__any_sync(kFull, close)) {
    if constexpr (!SIG) return false;
    // contested: the k best and all within the bound of the k-th (at most 32) in fp64, a lane each
    const float floor_v = __shfl_sync(kFull, v, a.k - 1) - gap;
    int n = a.k;
    while (last >= 8u && __uint_as_float(last & ~7u) >= floor_v) {
      if (n == 32) return false;
      take(n++, last);
      last = __reduce_max_sync(kFull, key[0]);
    }
    id = from + 32 * int(mine & 7u);
    const int rank = rank_fp64(lane < n ? __ldg(lr + id) : 0.f, sc.bias && lane < n ? __ldg(sc.bias + id) : 0.f,
                               id, n);
    if (lane < n && rank < a.k) ids[rank] = uint8_t(id);
  } else if (lane < a.k) {
    ids[lane] = uint8_t(id);
  }
#pragma unroll
  for (int i = 0; i < Q; ++i) pp[i] = fmaf(q[i], ti, pp[i]);
  return true;
}

template <int Q, bool SIG, bool ONE>
__global__ void __launch_bounds__(kTokThreads, Q >= 4 ? 1 : 2) route_scored_kernel(RouteArgs a, ScoreArgs sc) {
  // [warps][E] doubles of group scratch, then [warps][E] probability sums, then the counts
  // [k][4][E]
  extern __shared__ double s_dyn[];
  __shared__ float s_z[kWarps];
  __shared__ float s_sum[kThreads];  // sum of exp(l - top), later logsumexp^2
  __shared__ float s_top[kThreads];  // the largest logit of general tokens, 0 of the others
  __shared__ __align__(8) uint8_t s_id[kThreads * kMaxK];
  __shared__ uint8_t s_rk[kThreads * kMaxK];
  __shared__ float s_w[ONE ? kThreads * kMaxK : 1];  // the choices' weights
  const int c = blockIdx.x;
  const int g = c / a.n_cpg, cc = c % a.n_cpg;
  const int t0 = g * a.Sg + cc * kThreads;
  const int nt = min(kThreads, a.Sg - cc * kThreads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = a.E, k = a.k;
  pdl_wait();
  pdl_trigger();
  if (c == 0 && tid == 0) *a.done = 0u;  // ticket counter of route_scan_kernel

  float l[Q];
  auto fetch = [&](int i) {
    const float* lr = a.logits + int64_t(t0 + i) * E;
#pragma unroll
    for (int x = 0; x < Q; ++x) l[x] = lane + 32 * x < E ? __ldg(lr + lane + 32 * x) : -1e30f;
  };
  if (warp < nt) fetch(warp);  // the first token, beside the biases
  float b[Q];
  float bmin = INFINITY, bmax = -INFINITY;
  bool bias_bad = false;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    const int e = lane + 32 * i;
    b[i] = 0.f;
    if (e < E) {
      if (sc.bias) b[i] = __ldg(sc.bias + e);
      if (!isfinite(b[i])) bias_bad = true;
      bmin = fminf(bmin, b[i]);
      bmax = fmaxf(bmax, b[i]);
    }
  }
  bias_bad = __any_sync(kFull, bias_bad);
  if (bias_bad && tid == 0) atomicOr(a.status, kStatusNonfinite);
  bmin = -warp_max(-bmin);
  bmax = warp_max(bmax);
#pragma unroll
  for (int i = 0; i < Q; ++i)  // an expert's key is never below 8, no expert's is its slot
    b[i] = lane + 32 * i < E ? (b[i] - bmin) + 1e-30f : 0.f;
  const float brange = bmax - bmin;
  if (!(brange < 1e30f)) bias_bad = true;  // the shifted biases could overflow (no error)
  double* scratch = s_dyn + size_t(warp) * E;
  float pp[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) pp[i] = 0.f;
  for (int i = warp; i < nt; i += kTokWarps) {
    const float* lr = a.logits + int64_t(t0 + i) * E;
    if (i != warp) fetch(i);
    float s;
    if (!bias_bad && token_fast<Q, SIG>(l, b, brange, lr, a, sc, reinterpret_cast<float*>(scratch), pp,
                                        s_id + i * kMaxK, s)) {
      if (lane == 0) {
        s_sum[i] = s;
        s_top[i] = 0.f;
      }
    } else {
      float q[Q];
      bool bad = false;
#pragma unroll
      for (int x = 0; x < Q; ++x) {
        const bool in = lane + 32 * x < E;
        if (in && !isfinite(l[x])) bad = true;
        if (!in || !isfinite(l[x])) l[x] = -INFINITY;
      }
      if (bad) atomicOr(a.status, kStatusNonfinite);
      __syncwarp();
      float m;
      const int id = token_general<Q>(l, a, sc, scratch, q, m, s);
#pragma unroll
      for (int x = 0; x < Q; ++x) pp[x] += q[x];
      if (lane < k) s_id[i * kMaxK + lane] = uint8_t(id);
      if (lane == 0) {
        s_sum[i] = s;
        s_top[i] = m;
      }
    }
  }
  __syncthreads();
  // the weights: 8 lanes a token, lane j < k its choice j, from accurate exponentials: renormalised
  // ones of the choices' logits less their largest (they cannot all underflow), softmax ones of
  // l - top - log(sum), the largest logit taken off first (l less the rounded logsumexp would carry
  // half a step of it, 4e-3 of the weight at an offset of 1e5)
  for (int x = tid; x < kThreads * kMaxK; x += kTokThreads) {
    const int i = x >> 3, j = x & 7;
    const bool on = i < nt && j < k;
    float ls = -INFINITY, top = 0.f, log_sum = 0.f;
    int id = 0;
    if (i < nt) {
      top = s_top[i];
      log_sum = s_sum[i] > 0.f ? logf(s_sum[i]) : 0.f;
    }
    if (on) {
      id = int(s_id[i * kMaxK + j]);
      ls = __ldg(a.logits + int64_t(t0 + i) * E + id);
      if (!isfinite(ls) || (sc.bias && !isfinite(__ldg(sc.bias + id)))) ls = -INFINITY;
    }
    float w;
    if (sc.renorm) {
      float most = SIG ? fminf(ls, 0.f) : ls;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, off));
      if (!(most > -INFINITY)) most = 0.f;
      w = SIG ? sigmoid_shifted(ls, most) : (ls > -INFINITY ? expf(ls - most) : 0.f);
      float tot = w;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) tot += __shfl_xor_sync(kFull, tot, off);
      w = tot > 0.f ? w / tot : 0.f;
    } else {
      w = SIG ? sigmoid_shifted(ls, 0.f) : (ls > -INFINITY ? expf((ls - top) - log_sum) : 0.f);
    }
    if (on) {
      a.expert_id[int64_t(t0 + i) * k + j] = id;
      if (ONE) s_w[i * kMaxK + j] = w * sc.scale;
      else a.gate[int64_t(t0 + i) * k + j] = w * sc.scale;
    }
    // the token's logsumexp^2, kept for the sum below
    __syncwarp();
    if (i < nt && j == 0) s_sum[i] = (top + log_sum) * (top + log_sum);
  }
  __syncthreads();  // the group scratch is free
  float* s_pp = reinterpret_cast<float*>(s_dyn);
#pragma unroll
  for (int i = 0; i < Q; ++i)
    if (lane + 32 * i < E) s_pp[warp * E + lane + 32 * i] = pp[i];
  if (tid < kThreads) {
    const float z = warp_sum(tid < nt ? s_sum[tid] : 0.f);
    if (lane == 0) s_z[warp] = z;
  }
  __syncthreads();
  float psum = 0.f;  // of expert tid
  if (tid < E) {
#pragma unroll
    for (int w = 0; w < kTokWarps; ++w) psum += s_pp[w * E + tid];
    if (!ONE) a.ppart[size_t(c) * E + tid] = psum;
  }
  float sz = 0.f;
  if (tid == 0) {
    for (int w = 0; w < kWarps; ++w) sz += s_z[w];
    if (!ONE) a.zpart[c] = sz;
  }
  __syncthreads();

  // rank of each choice among the chunk's earlier ones of the same (j, e): the first
  // kThreads threads hold a token each; counts per (j, warp, e), one scan over the warps
  int* s_cnt = reinterpret_cast<int*>(s_dyn);
  const int nw = (nt + 31) >> 5;  // of the kWarps groups of 32 tokens, those that hold any
  for (int x = tid; x < k * nw * E; x += kTokThreads) s_cnt[x] = 0;
  __syncthreads();
  const unsigned lt_mask = (1u << lane) - 1u;
  if (warp < nw) {
    for (int j = 0; j < k; ++j) {
      const bool on = tid < nt;
      const int e = on ? int(s_id[tid * kMaxK + j]) : -1;
      const unsigned peers = __match_any_sync(kFull, on ? e : 1024 + lane);
      const int rk = __popc(peers & lt_mask);
      s_rk[tid * kMaxK + j] = uint8_t(rk);
      if (on && rk == 0) s_cnt[(j * nw + warp) * E + e] = __popc(peers);
    }
  }
  __syncthreads();
  if constexpr (!ONE) {
    for (int x = tid; x < E; x += kTokThreads) {  // choice ranks in order: expert x's columns
      int all = 0;
      for (int j = 0; j < k; ++j) {
        int run = 0;
        for (int w = 0; w < nw; ++w) {
          int* cw = s_cnt + (j * nw + w) * E + x;
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
      a.rank[size_t(t0) * k + x] = s_cnt[(j * nw + (i >> 5)) * E + e] + int(s_rk[i * kMaxK + j]);
    }
  } else {
    // the whole batch is here: slots, offsets, rows and losses as the scan and finalize
    // kernels form them
    __shared__ int s_first[kMaxE], s_wsum[kMaxE / 32];
    __shared__ float s_aux[kMaxE / 32];
    int all = 0, kept = 0;
    if (tid < E) {
      for (int j = 0; j < k; ++j)
        for (int w = 0; w < nw; ++w) {
          int* cw = s_cnt + (j * nw + w) * E + tid;
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
      const int slot = s_cnt[(j * nw + (i >> 5)) * E + e] + int(s_rk[i * kMaxK + j]);
      const bool in = a.C < 0 || slot < a.C;
      const int row = in ? s_first[e] + slot : -1;
      const float w = s_w[i * kMaxK + j];
      a.pos[x] = in ? slot : -1;
      a.row[x] = row;
      a.drop[x] = in ? MOE_KEPT : MOE_DROP_CAPACITY;
      if (in) {
        a.token_of[row] = i;
        a.w_perm[row] = w;
      }
      a.gate[x] = in ? w : 0.f;
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
// with ca = aux_coef E / (G S_g). 1 - s = 1 / (1 + exp(l)), so it keeps its precision where s is
// close to 1. One exponential an expert serves all of it: x = exp(l) where the logits lie within
// +-80 (their sum then neither overflows nor vanishes), s = x / (1 + x); else exp(l - max) for the
// softmax and shifted sigmoids apart. 16384 x 256: 15 us (with three exponentials an expert 29);
// 62 % of the issue slots are taken; memory (8 S E bytes) would take 5 us.
constexpr int kBwdWarps = 8, kBwdTokens = 2;  // warps a CTA, consecutive tokens a warp
// A lane without an expert brings exp(-80) into the sums (a select an expert to leave it out took 1 us
// more): of a sum of exponentials above this, all 255 of them together are less than 5e-9. Below it
// the token takes the general form, whose sums hold experts alone.
constexpr float kFewest = 1e-24f;

template <int Q, bool SIG>
__global__ void __launch_bounds__(32 * kBwdWarps, 4)
    route_scored_bwd_kernel(const float* __restrict__ logits, const int32_t* __restrict__ expert_id,
                            const int32_t* __restrict__ row, const int32_t* __restrict__ counts_routed,
                            const float* __restrict__ dgate, const float* __restrict__ gpart,
                            int n_tiles, int S, int G, int E, int k, ScoreArgs sc, float aux_coef,
                            float z_coef, float* __restrict__ dlogits,
                            __nv_bfloat16* __restrict__ dlb, int Ep) {
  __shared__ float s_dl[kBwdWarps][32 * Q];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = (int64_t(blockIdx.x) * kBwdWarps + warp) * kBwdTokens;
  const int Sg = S / G;
  const float ca = aux_coef * float(E) / (float(G) * float(Sg)) / (float(Sg) * float(k));
  const float cz = z_coef * 2.f / float(S);
  float* sd = s_dl[warp];
  float f[Q];  // ca times the routed counts of the token's group
  int group = -1;
  for (int64_t t = first; t < first + kBwdTokens && t < S; ++t) {
    const float* lr = logits + t * E;
    float l[Q], p[Q], q[Q], om[Q];  // p: softmax; q: normalised scores; om: 1 - s
    bool plain = true;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < E ? __ldg(lr + e) : -80.f;  // no expert (f = 0): see kFewest
      plain = plain && fabsf(l[i]) <= 80.f;  // false for NaN too
    }
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
    if (aux_coef != 0.f && int(t / Sg) != group) {
      group = int(t / Sg);
#pragma unroll
      for (int i = 0; i < Q; ++i)
        f[i] = lane + 32 * i < E ? ca * float(counts_routed[int64_t(group) * E + lane + 32 * i]) : 0.f;
    }
    float s = 0.f, tot = 0.f, m = 0.f, lse;
    bool fast = __all_sync(kFull, plain);
    if (fast) {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const float x = expf(l[i]);
        p[i] = x;
        s += x;
        if constexpr (SIG) {
          om[i] = rcp_approx(1.f + x);
          q[i] = x * om[i];
          tot += q[i];
        }
      }
      s = warp_sum(s);
      lse = logf(s);
      fast = s > kFewest;
    }
    if (!fast) {
      m = -INFINITY;
      s = tot = 0.f;
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        l[i] = lane + 32 * i < E ? __ldg(lr + lane + 32 * i) : -INFINITY;
        if (!isfinite(l[i])) l[i] = -INFINITY;
        m = fmaxf(m, l[i]);
      }
      m = warp_max(m);
      const bool any = m > -INFINITY;
      if (!any) m = 0.f;
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        p[i] = expf(l[i] - m);
        s += p[i];
        if constexpr (SIG) {
          om[i] = l[i] > -INFINITY ? sigmoid_shifted(-l[i], 0.f) : 1.f;
          q[i] = sigmoid_shifted(l[i], fminf(m, 0.f));
          tot += q[i];
        }
      }
      s = warp_sum(s);
      lse = any ? m + logf(s) : 0.f;
    }
    const float inv = s > 0.f ? rcp_approx(s) : 0.f;
    if constexpr (SIG) tot = warp_sum(tot);
    const float ti = SIG ? (tot > 0.f ? rcp_approx(tot) : 0.f) : inv;
    // the weights of the choices (unscaled; lanes j < 8, the others idle along)
    float w, inner = 0.f;
    if (sc.renorm) {
      float top = SIG ? fminf(lsel, 0.f) : lsel;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
      if (!(top > -INFINITY)) top = 0.f;
      w = SIG ? sigmoid_shifted(lsel, top) : (lsel > -INFINITY ? expf(lsel - top) : 0.f);
      float all = w;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) all += __shfl_xor_sync(kFull, all, off);
      w = all > 0.f ? w / all : 0.f;
    } else {
      w = SIG ? sigmoid_shifted(lsel, 0.f) : (lsel > -INFINITY ? expf(lsel - m) * inv : 0.f);
    }
    if (sc.renorm || !SIG) {
      inner = w * dg;
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) inner += __shfl_xor_sync(kFull, inner, off);
      inner = __shfl_sync(kFull, inner, 0);
    }
    float dsel = sc.scale * w * ((sc.renorm ? dg - inner : dg) * (SIG ? sigmoid_shifted(-lsel, 0.f) : 1.f));
    if (!(lsel > -INFINITY)) dsel = 0.f;
    // the dense part: the losses' gradients (and the un-normalised softmax weights' common one)
    const float cp = cz * lse * inv - (!SIG && !sc.renorm ? sc.scale * inner * inv : 0.f);
    float fq = 0.f;
    if (aux_coef != 0.f) {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        q[i] = (SIG ? q[i] : p[i]) * ti;
        fq = fmaf(f[i], q[i], fq);
      }
      fq = warp_sum(fq);
    }
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      float d = p[i] * cp;
      if (aux_coef != 0.f) d = fmaf(SIG ? q[i] * om[i] : q[i], f[i] - fq, d);
      sd[lane + 32 * i] = d;
    }
    __syncwarp();
    if (id >= 0) sd[id] += dsel;  // the choices are distinct experts
    __syncwarp();
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const int e = lane + 32 * i;
      const float d = sd[e];
      if (e < E) dlogits[t * E + e] = d;
      if (dlb && e < Ep) dlb[t * Ep + e] = __float2bfloat16_rn(e < E ? d : 0.f);
    }
    __syncwarp();
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
  const bool one = L.n_chunks == 1 && !d, sig = sc.score == MOE_SCORE_SIGMOID;
  auto launch = [&](auto kern) -> int {
    // at most 32 KB (E <= 256, k <= 8)
    const size_t dyn = std::max(size_t(kTokWarps) * c.E * sizeof(double), size_t(c.k) * kWarps * c.E * 4);
    return launch_kernel(kern, dim3(unsigned(L.n_chunks)), dim3(kTokThreads), dyn, st, a,
                         score_args(sc, select_bias));
  };
  auto go = [&](auto q) -> int {
    constexpr int Q = decltype(q)::value;
    if (sig) return one ? launch(route_scored_kernel<Q, true, true>) : launch(route_scored_kernel<Q, true, false>);
    return one ? launch(route_scored_kernel<Q, false, true>) : launch(route_scored_kernel<Q, false, false>);
  };
  const int rc = c.E <= 32    ? go(std::integral_constant<int, 1>{})
                 : c.E <= 64  ? go(std::integral_constant<int, 2>{})
                 : c.E <= 128 ? go(std::integral_constant<int, 4>{})
                              : go(std::integral_constant<int, 8>{});
  if (rc != MOE_OK || one) return rc;
  return launch_scan_finalize(c, a, d, st);
}

int launch_route_scored_backward(const moe_config_t& c, const moe_score_t& sc, const float* logits,
                                 const moe_route_out_t& r, const float* dgate, const float* gpart,
                                 int n_tiles, float aux_coef, float z_coef, float* dlogits, void* dlb,
                                 int Ep, cudaStream_t st) {
  const int64_t per = kBwdWarps * kBwdTokens;
  auto launch = [&](auto kern) -> int {
    return launch_kernel(kern, dim3(unsigned((c.S + per - 1) / per)), dim3(32 * kBwdWarps), 0, st, logits,
                         static_cast<const int32_t*>(r.expert_id), static_cast<const int32_t*>(r.row),
                         static_cast<const int32_t*>(r.counts_routed), dgate, gpart, n_tiles, c.S, c.G, c.E, c.k,
                         score_args(sc, nullptr), aux_coef, z_coef, dlogits, static_cast<__nv_bfloat16*>(dlb), Ep);
  };
  auto go = [&](auto q) -> int {
    constexpr int Q = decltype(q)::value;
    return sc.score == MOE_SCORE_SIGMOID ? launch(route_scored_bwd_kernel<Q, true>)
                                         : launch(route_scored_bwd_kernel<Q, false>);
  };
  // (dlb's columns go up to E rounded up to 64)
  const int cols = dlb ? Ep : c.E;
  return cols <= 32    ? go(std::integral_constant<int, 1>{})
         : cols <= 64  ? go(std::integral_constant<int, 2>{})
         : cols <= 128 ? go(std::integral_constant<int, 4>{})
                       : go(std::integral_constant<int, 8>{});
}

}  // namespace moe
