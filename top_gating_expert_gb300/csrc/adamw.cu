// One AdamW step over many tensors, and the global norm of many gradients.
//
//   g' = g c                      c = min(1, max_norm / (norm + 1e-6)), or 1
//   m  = b1 m + (1 - b1) g'       v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// element by element, bound by memory: an fp32 parameter with fp32 moments moves 28 bytes (30 with
// its bf16 copy), with 8-bit moments 16 (18). 2^28 fp32 elements: 1147 us in 32 bits (6.55 TB/s, 0.98 of the
// copy rate), 1245 with the copy; in 8 bits 809 (nearest codes; 5.3 TB/s) and 919 (random): 100 instructions an element,
// 72 % of the issue slots, beside 61 % of DRAM's rate. The values of the codes: 444 us (6.0 TB/s); the norm 172 us
// (bf16 92). The tensors' table travels as a kernel argument (no
// copy to the device, and a captured graph holds it), in the smallest of three sizes that takes it;
// persistent CTAs walk chunks of 2048 elements over all tensors, a warp 256 of them, and find a
// chunk's tensor by halving.
//
// The moments of all tensors lie in one buffer each, every tensor from a multiple of 256 on. In 8
// bits, 256 elements share a scale s, their largest |m| (or sqrt(v)), and a code c stands for
//   m ~ sign(c) (c / 127)^2 s,     sqrt(v) ~ (c / 255)^2 s:
// quadratic steps, fine near zero. With y = 127^2 |m| / s the code is the k with k^2 <= y < (k + 1)^2,
// or k + 1 where y - k^2 > r (2k + 1): r = 1/2 takes the nearer value, a random r of (0, 1) makes the
// value's expectation y itself, so that changes much smaller than a step are not lost (b2 = 0.999
// moves v by 0.1 % a step, codes are 0.8 % apart at best). r comes from a hash of seed, step and
// place. No sqrt(v) above 0 goes to code 0: m / sqrt(v) would grow without bound. What keeps its mean is the root: v
// itself is high by the root's variance, in a run of steps by about 1 / c of itself at code c (normal gradients, beta2 0.95
// and 0.999 alike: 13 % at code 8, 1 % at 81), and 1 / sqrt(v), by which a step is as long, by about 0.3 / c.
// The update takes the moments before they are rounded. Operations on the way to a code are
// rounded one by one (no fused multiply-add), so the codes are a function of the formula alone.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "elem.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlock = 256;                // elements that share a scale: a warp's, 8 a lane
constexpr int kChunk = kWarps * kBlock;    // elements of a CTA's step
constexpr int kNormChunk = 8192;           // elements of a CTA's step of the norm
constexpr int kNormSlots = 2048;           // partial sums of the norm: CTAs at most
constexpr float kMLevels = 127.f * 127.f, kVLevels = 255.f * 255.f;

struct Tensor {
  void* p;
  const void* g;
  void* copy;
  int64_t n, first, chunk0;  // elements, place in the moments, chunks before it
  float decay, wd;           // 1 - lr wd (lr by value), wd (lr on the device)
  int p_bf16, g_bf16, vec;   // vec: 4 elements an access everywhere
};
template <int CAP>
struct Table {
  Tensor t[CAP];
};

struct StepArgs {
  int n, last;  // last: the launch that advances the clock
  int64_t chunks;
  void *m, *v;
  float *m_scale, *v_scale;
  double* clock;  // t, b1^t, b2^t of the steps made
  const float* lr_dev;
  const float* norm;
  unsigned* ticket;
  double beta1, beta2;
  float lr, b1, c1, b2, c2, eps, max_norm;
  int64_t seed;  // < 0: codes of the nearest values
};

// The tensor of a chunk: the last one with chunk0 <= chunk.
template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP>& tab, int n, int64_t chunk) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.t[mid].chunk0 <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Four elements i .. i + 3 as one access
__device__ __forceinline__ float4 load4(const void* base, int bf16, int64_t i) {
  if (!bf16) return __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(base) + i));
  const uint2 w = __ldcs(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + i));
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(void* base, int bf16, int64_t i, const float (&f)[4]) {
  if (!bf16) {
    __stcs(reinterpret_cast<float4*>(static_cast<float*>(base) + i), make_float4(f[0], f[1], f[2], f[3]));
  } else {
    __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    __stcs(reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + i),
           make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b)));
  }
}

__device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x9E3779B1u;
  h ^= h >> 15;
  h *= 0x85157AF5u;
  return h ^ (h >> 16);
}

// Conversions between small whole numbers and fp32 by the number's place in a float's mantissa (a
// conversion instruction takes the slow unit, which the square roots fill).
__device__ __forceinline__ float byte_bits(uint32_t w, int k) {  // 2^23 + byte k of w
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540u | k));
}
// the low bytes of four words
__device__ __forceinline__ uint32_t pack_bytes(const uint32_t (&w)[4]) {
  return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}
// the hardware's root (within 2^-21): with denormals, or with those taken as 0
__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sqrt_approx_ftz(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// the largest magnitude of three (NaN if one is)
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Codes. For y >= 0 (in units of the scale, times the levels) the code is k + 1 where t = y - k^2 > r (2k + 1),
// else k, for the k with k^2 <= y < (k + 1)^2; f = 2^16 r. k comes from the hardware's root plus
// 2^-14 less 1/2, rounded: it is never less (the root is within 2^-23, the sum within 2^-17), and next to the
// following square k + 1 (t < 0).
constexpr float kToFloor = -0.5f + 0x1p-14f, kMagic = 12582912.f;  // 1.5 * 2^23
__device__ __forceinline__ f32x2 floor_root2(f32x2 y) {
  const float2 f = unpack2(y);
  return add2(add2(add2(pack2(sqrt_approx_ftz(f.x), sqrt_approx_ftz(f.y)), set2(kToFloor)), set2(kMagic)), set2(-kMagic));
}
__device__ __forceinline__ f32x2 limit2(const float (&f)[2], f32x2 k) {  // r (2k + 1), rounded once
  return mul2(pack2(f[0], f[1]), fma2(k, set2(0x1p-15f), set2(0x1p-16f)));
}
// the codes of two exact y
__device__ __forceinline__ void exact_codes(const float (&y)[2], const float (&f)[2], float (&code)[2]) {
  const float2 k2 = unpack2(floor_root2(pack2(y[0], y[1])));
  float k[2] = {k2.x, k2.y}, t[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    t[i] = fmaf(-k[i], k[i], y[i]);
    if (t[i] < 0.f) {
      k[i] -= 1.f;
      t[i] = fmaf(-k[i], k[i], y[i]);
    }
  }
  const float2 lim = unpack2(limit2(f, pack2(k[0], k[1])));
  code[0] = t[0] > lim.x ? k[0] + 1.f : k[0];
  code[1] = t[1] > lim.y ? k[1] + 1.f : k[1];
}
// The same without the correction of k and for y off by up to y 2^-21: `margin` becomes negative where a code may be
// another one (t not safely above 0, where k and the limit may belong to the next square, or close to the limit).
// Not for `top`, the block's largest value, whose y is next to a square always, as long as r does not come within 2^-17
// of 1: its code is then the highest (y is at most two roundings, 2^-23, below the highest square).
__device__ __forceinline__ void near_codes(f32x2 y, const float (&f)[2], float v0, float v1, float top, float (&code)[2],
                                           float& margin) {
  const f32x2 k2 = floor_root2(y);
  const float2 yf = unpack2(y), k = unpack2(k2), lim = unpack2(limit2(f, k2));
  const float t0 = fmaf(-k.x, k.x, yf.x), t1 = fmaf(-k.y, k.y, yf.y);
  code[0] = k.x;
  code[1] = k.y;
  if (t0 > lim.x) code[0] += 1.f;
  if (t1 > lim.y) code[1] += 1.f;
  if (v0 != top || f[0] > 65535.f) margin = min3(margin, fmaf(yf.x, -0x1p-21f, t0), fmaf(yf.x, -0x1p-21f, fabsf(t0 - lim.x)));
  if (v1 != top || f[1] > 65535.f) margin = min3(margin, fmaf(yf.y, -0x1p-21f, t1), fmaf(yf.y, -0x1p-21f, fabsf(t1 - lim.y)));
}
__device__ __forceinline__ float v_code(float c, float y) {  // 0 for 0 alone, 255 at most
  return fminf(fmaxf(c, __saturatef(y * 0x1p126f)), 255.f);
}

// A block's scale from the bits of its largest magnitude: NaN where one is not finite, 0 below 2^-100
// (its values are then 0); and levels / scale.
__device__ __forceinline__ void block_scale(uint32_t bits, float levels, float& s, float& inv) {
  const float top = __uint_as_float(bits);
  s = bits >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : (top >= 0x1p-100f ? top : 0.f);
  inv = s == 0.f ? 0.f : __fdiv_rn(levels, s);
}

// What all blocks of a step share.
struct Shared {
  float size, rs, coef;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t), the clip factor
  uint32_t key;
};

// A warp's 256 elements e0 .. of tensor x, places s0 .. of the moments, 8 a lane. FULL: all of them exist, in
// accesses of four elements; else (a tensor's end, rows on no boundary) one by one, neighbouring lanes on
// neighbouring elements (12.7 M bf16 parameters and gradients on no boundary: 56 us, with four in a row a
// lane 80). P16, G16: p and g in
// bf16.
template <int BITS, bool FULL, bool P16, bool G16>
__device__ __forceinline__ void adamw_block(const Tensor& x, const StepArgs& a, const Shared& sh, float decay, int64_t e0,
                                            int64_t s0, int valid_) {
  const int lane = threadIdx.x & 31;
  const int valid = FULL ? kBlock : valid_;
  constexpr int p16 = P16, g16 = G16;
  // the place of a lane's e-th element, and four of them (4 q ..) from and to memory
  auto place_of = [&](int e) { return FULL ? 128 * (e / 4) + 4 * lane + (e & 3) : 32 * e + lane; };
  auto load = [&](const void* base, int bf16, int64_t from, int q) {
    if constexpr (FULL) return load4(base, bf16, from + place_of(4 * q));
    float f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = place_of(4 * q + k);
      f[k] = 0.f;
      if (i < valid)
        f[k] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(base)[from + i])
                    : static_cast<const float*>(base)[from + i];
    }
    return make_float4(f[0], f[1], f[2], f[3]);
  };
  auto store = [&](void* base, int bf16, int64_t from, int q, const float (&f)[4]) {
    if constexpr (FULL) {
      store4(base, bf16, from + place_of(4 * q), f);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = place_of(4 * q + k);
        if (i >= valid) continue;
        if (bf16) static_cast<__nv_bfloat16*>(base)[from + i] = __float2bfloat16_rn(f[k]);
        else static_cast<float*>(base)[from + i] = f[k];
      }
    }
  };
  // codes: every block of theirs is whole
  auto load_codes = [&](const void* base, int q) {
    const uint8_t* c = static_cast<const uint8_t*>(base) + s0;
    if constexpr (FULL) return __ldcs(reinterpret_cast<const uint32_t*>(c + place_of(4 * q)));
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) w |= uint32_t(c[place_of(4 * q + k)]) << (8 * k);
    return w;
  };
  auto store_codes = [&](void* base, int q, uint32_t w) {
    uint8_t* c = static_cast<uint8_t*>(base) + s0;
    if constexpr (FULL) {
      __stcs(reinterpret_cast<uint32_t*>(c + place_of(4 * q)), w);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) c[place_of(4 * q + k)] = uint8_t(w >> (8 * k));
    }
  };
  const float size = sh.size, rs = sh.rs, coef = sh.coef;
  const uint32_t key = sh.key;
  float4 pv[2], gv[2], mv[2], vv[2];
  uint32_t mc[2], vc[2];
  float ms = 0.f, vs = 0.f;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    gv[q] = load(x.g, g16, e0, q);
    pv[q] = load(x.p, p16, e0, q);
    if constexpr (BITS == 32) {
      mv[q] = load(a.m, 0, s0, q);
      vv[q] = load(a.v, 0, s0, q);
    } else {
      mc[q] = load_codes(a.m, q);
      vc[q] = load_codes(a.v, q);
    }
  }
  if constexpr (BITS == 8) {
    ms = __fmul_rn(a.m_scale[s0 / kBlock], 1.f / kMLevels);
    vs = __fmul_rn(a.v_scale[s0 / kBlock], 1.f / kVLevels);
  }
  // What does not exist reads as 0 (the codes behind a tensor's end are), and its moments stay 0.
  float m[8], v[8];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float g4[4] = {gv[q].x, gv[q].y, gv[q].z, gv[q].w};
    const float p4[4] = {pv[q].x, pv[q].y, pv[q].z, pv[q].w};
    float m4[4], v4[4], out[4];
    if constexpr (BITS == 32) {
      m4[0] = mv[q].x; m4[1] = mv[q].y; m4[2] = mv[q].z; m4[3] = mv[q].w;
      v4[0] = vv[q].x; v4[1] = vv[q].y; v4[2] = vv[q].z; v4[3] = vv[q].w;
    }
    const uint32_t flip = BITS == 8 ? mc[q] ^ 0x80808080u : 0u;  // signed bytes from 0 on
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      f32x2 m2, v2;
      if constexpr (BITS == 32) {
        m2 = pack2(m4[k], m4[k + 1]);
        v2 = pack2(v4[k], v4[k + 1]);
      } else {
        const float2 cm = unpack2(add2(pack2(byte_bits(flip, k), byte_bits(flip, k + 1)), set2(-8388736.f)));
        const f32x2 cv = add2(pack2(byte_bits(vc[q], k), byte_bits(vc[q], k + 1)), set2(-8388608.f));
        m2 = mul2(pack2(cm.x * fabsf(cm.x), cm.y * fabsf(cm.y)), set2(ms));
        const f32x2 u2 = mul2(mul2(cv, cv), set2(vs));
        v2 = mul2(u2, u2);
      }
      // Every product and sum of the moments is rounded by itself: the sums one by one, since the
      // assembler fuses a sum of pairs with a product of pairs in front of it
      const f32x2 g2 = mul2(pack2(g4[k], g4[k + 1]), set2(coef));
      const float2 bm = unpack2(mul2(m2, set2(a.b1))), gm = unpack2(mul2(g2, set2(a.c1)));
      const float2 bv = unpack2(mul2(v2, set2(a.b2))), gg = unpack2(mul2(mul2(g2, g2), set2(a.c2)));
      const float2 mf = make_float2(__fadd_rn(bm.x, gm.x), __fadd_rn(bm.y, gm.y));
      const float2 vf = make_float2(__fadd_rn(bv.x, gg.x), __fadd_rn(bv.y, gg.y));
      // the step takes the hardware's root and reciprocal: a few ulp of a step that is 10^-3 of p
      const float2 den = unpack2(fma2(pack2(sqrt_approx(vf.x), sqrt_approx(vf.y)), set2(rs), set2(a.eps)));
      const f32x2 step = mul2(mul2(pack2(mf.x, mf.y), pack2(rcp_approx(den.x), rcp_approx(den.y))), set2(-size));
      const float2 pn = unpack2(fma2(pack2(p4[k], p4[k + 1]), set2(decay), step));
      out[k] = pn.x;
      out[k + 1] = pn.y;
      const int e = 4 * q + k;
      m[e] = mf.x;
      m[e + 1] = mf.y;
      v[e] = vf.x;
      v[e + 1] = vf.y;
    }
    store(x.p, p16, e0, q, out);
    if (x.copy) store(x.copy, 1, e0, q, out);
    if constexpr (BITS == 32) {
      store(a.m, 0, s0, q, reinterpret_cast<const float(&)[4]>(m[4 * q]));
      store(a.v, 0, s0, q, reinterpret_cast<const float(&)[4]>(v[4 * q]));
    }
  }
  if constexpr (BITS == 8) {
    // bits of magnitudes compare as the magnitudes do, NaN above all; the root of the largest v is the
    // largest root
    float mt = max3_abs(m[0], m[1], m[2]), vt = max3_abs(v[0], v[1], v[2]);
    mt = max3_abs(mt, m[3], m[4]);
    vt = max3_abs(vt, v[3], v[4]);
    mt = max3_abs(mt, m[5], max3_abs(m[6], m[7], 0.f));
    vt = max3_abs(vt, v[5], max3_abs(v[6], v[7], 0.f));
    const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(mt));
    const uint32_t vb = __reduce_max_sync(0xffffffffu, __float_as_uint(vt));
    // one division for both: the lower lanes m's, the upper ones v's
    float s2, i2;
    block_scale(lane < 16 ? mb : __float_as_uint(__fsqrt_rn(__uint_as_float(vb))), lane < 16 ? kMLevels : kVLevels, s2, i2);
    const float im = __shfl_sync(0xffffffffu, i2, 0), iv = __shfl_sync(0xffffffffu, i2, 16);
    // The thresholds of element e, times 2^16: the halves of mix32(place ^ key), plus 1/2. In the place the bits of
    // the element in the lane are apart from the lane's, so the hash's first step is shared.
    const uint32_t x0 = uint32_t(s0 + place_of(0)) ^ (uint32_t(s0 >> 32) * 0x2545F491u) ^ key, x1 = x0 ^ (x0 >> 16);
    auto thresholds = [&](int e, float& fm, float& fv) {
      uint32_t h = (x1 ^ uint32_t(FULL ? 128 * (e / 4) + (e & 3) : 32 * e)) * 0x9E3779B1u;
      h = (h ^ (h >> 15)) * 0x85157AF5u;
      fm = __uint_as_float(__byte_perm(h ^ (h >> 16), 0x4B000000u, 0x7610u));
      fv = __uint_as_float(__byte_perm(h, 0x4B000000u, 0x7632u));
    };
    auto thresholds2 = [&](int e, float (&fm)[2], float (&fv)[2]) {
      float m0, m1, v0, v1;
      thresholds(e, m0, v0);
      thresholds(e + 1, m1, v1);
      const float2 a2 = unpack2(add2(pack2(m0, m1), set2(-8388607.5f))), b2 = unpack2(add2(pack2(v0, v1), set2(-8388607.5f)));
      fm[0] = a2.x; fm[1] = a2.y;
      fv[0] = b2.x; fv[1] = b2.y;
    };
    // roots of 2^24 v, which no denormal v is too small for; largest ones too large for it go the exact way
    const float iv12 = iv * 0x1p-12f;
    uint32_t wm[2], wv[2];
    float margin = vb >= 0x71800000u ? -1.f : 0.f;  // 2^100
    auto codes = [&](auto exact) {
      constexpr bool EXACT = decltype(exact)::value;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t bm[4], bv[4];
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const int e = 4 * q + k;
          float fm[2] = {32768.f, 32768.f}, fv[2] = {32768.f, 32768.f};
          if (a.seed >= 0) thresholds2(e, fm, fv);
          const float ym[2] = {__fmul_rn(fabsf(m[e]), im), __fmul_rn(fabsf(m[e + 1]), im)};
          float cm[2], cv[2], yv[2];
          if constexpr (!EXACT) exact_codes(ym, fm, cm);
          if constexpr (EXACT) {
            yv[0] = __fmul_rn(__fsqrt_rn(v[e]), iv);
            yv[1] = __fmul_rn(__fsqrt_rn(v[e + 1]), iv);
            exact_codes(yv, fv, cv);
          } else {
            const float2 up = unpack2(mul2(pack2(v[e], v[e + 1]), set2(0x1p24f)));
            const f32x2 y2 = mul2(pack2(sqrt_approx_ftz(up.x), sqrt_approx_ftz(up.y)), set2(iv12));
            const float2 f = unpack2(y2);
            yv[0] = f.x;
            yv[1] = f.y;
            near_codes(y2, fv, v[e], v[e + 1], __uint_as_float(vb), cv, margin);
          }
          // whole numbers in the mantissa's low byte; after a NaN scale any
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if constexpr (!EXACT) bm[k + i] = __float_as_uint(copysignf(fminf(cm[i], 127.f), m[e + i]) + kMagic);
            bv[k + i] = __float_as_uint(v_code(cv[i], yv[i]) + kMagic);
          }
        }
        if constexpr (!EXACT) wm[q] = pack_bytes(bm);
        wv[q] = pack_bytes(bv);
      }
    };
    codes(std::false_type{});
    // some code of v is near a border (about one block of twenty): the block's from correctly rounded roots
    if (__any_sync(0xffffffffu, margin < 0.f)) codes(std::true_type{});
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      store_codes(a.m, q, wm[q]);
      store_codes(a.v, q, wv[q]);
    }
    if ((lane & 15) == 0) (lane == 0 ? a.m_scale : a.v_scale)[s0 / kBlock] = s2;
  }
}

template <int BITS, int CAP>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ Table<CAP> tab, const StepArgs a) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const float lr = a.lr_dev ? __ldg(a.lr_dev) : a.lr;
  Shared sh;
  sh.size = __fdiv_rn(lr, float(1.0 - a.clock[1] * a.beta1));
  sh.rs = __fdiv_rn(1.f, __fsqrt_rn(float(1.0 - a.clock[2] * a.beta2)));
  sh.coef = 1.f;
  if (a.norm) {
    sh.coef = __fdiv_rn(a.max_norm, __fadd_rn(__ldg(a.norm), 1e-6f));
    if (sh.coef > 1.f) sh.coef = 1.f;  // NaN stays
  }
  sh.key = 0;
  if (BITS == 8 && a.seed >= 0) sh.key = mix32(uint32_t(a.seed) + 0x632BE5ABu * uint32_t(int64_t(a.clock[0] + 1.0)));

  int at = 0;
  int64_t end = 0;  // the first chunk that is not tensor at's
  for (int64_t chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    if (chunk >= end) {
      at = tensor_of(tab, a.n, chunk);
      end = at + 1 < a.n ? tab.t[at + 1].chunk0 : a.chunks;
    }
    const Tensor& x = tab.t[at];
    const int64_t e0 = (chunk - x.chunk0) * kChunk + warp * kBlock;
    if (e0 >= x.n) continue;  // the whole warp
    const int64_t s0 = x.first + e0;
    const int valid = int(min(int64_t(kBlock), x.n - e0));
    const float decay = a.lr_dev ? fmaf(-lr, x.wd, 1.f) : x.decay;
    const bool full = valid == kBlock && x.vec;
    switch ((full ? 4 : 0) + (x.p_bf16 ? 2 : 0) + (x.g_bf16 ? 1 : 0)) {  // the same for the whole warp
      case 0: adamw_block<BITS, false, false, false>(x, a, sh, decay, e0, s0, valid); break;
      case 1: adamw_block<BITS, false, false, true>(x, a, sh, decay, e0, s0, valid); break;
      case 2: adamw_block<BITS, false, true, false>(x, a, sh, decay, e0, s0, valid); break;
      case 3: adamw_block<BITS, false, true, true>(x, a, sh, decay, e0, s0, valid); break;
      case 4: adamw_block<BITS, true, false, false>(x, a, sh, decay, e0, s0, valid); break;
      case 5: adamw_block<BITS, true, false, true>(x, a, sh, decay, e0, s0, valid); break;
      case 6: adamw_block<BITS, true, true, false>(x, a, sh, decay, e0, s0, valid); break;
      case 7: adamw_block<BITS, true, true, true>(x, a, sh, decay, e0, s0, valid); break;
    }
  }
  if (!a.last) return;
  // every CTA has read the clock by its turn here; the last one advances it
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(a.ticket, 1u) == gridDim.x - 1) {
      *a.ticket = 0u;
      a.clock[0] += 1.0;
      a.clock[1] *= a.beta1;
      a.clock[2] *= a.beta2;
    }
  }
}

// The moments' 32-bit values from their codes, blocks of 256.
__global__ void __launch_bounds__(kThreads)
    adamw_values_kernel(const int8_t* __restrict__ mc, const uint8_t* __restrict__ vc, const float* __restrict__ m_scale,
                        const float* __restrict__ v_scale, int64_t n, float* __restrict__ m, float* __restrict__ v) {
  pdl_wait();
  pdl_trigger();
  for (int64_t i = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 4; i < n; i += int64_t(gridDim.x) * kThreads * 4) {
    const uint32_t wm = __ldcs(reinterpret_cast<const uint32_t*>(mc + i)) ^ 0x80808080u;
    const uint32_t wv = __ldcs(reinterpret_cast<const uint32_t*>(vc + i));
    const float ms = __fmul_rn(__ldg(m_scale + i / kBlock), 1.f / kMLevels);
    const float vs = __fmul_rn(__ldg(v_scale + i / kBlock), 1.f / kVLevels);
    float fm[4], fv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = byte_bits(wm, k) - 8388736.f, b = byte_bits(wv, k) - 8388608.f;
      fm[k] = __fmul_rn(a * fabsf(a), ms);
      const float u = __fmul_rn(b * b, vs);
      fv[k] = __fmul_rn(u, u);
    }
    __stcs(reinterpret_cast<float4*>(m + i), make_float4(fm[0], fm[1], fm[2], fm[3]));
    __stcs(reinterpret_cast<float4*>(v + i), make_float4(fv[0], fv[1], fv[2], fv[3]));
  }
}

struct NormArgs {
  int n, first, last;  // first: the sum starts here; last: the norm is written
  int64_t chunks;
  float* out;
  float* part;     // [kNormSlots]
  double* total;
  unsigned* ticket;
};

// Sum of squares of all elements: fp32 within a thread (a lane's elements of one chunk first), a fixed
// tree over a CTA, fp64 over the CTAs in the last one to finish; launches add up in order.
template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) grad_norm_kernel(const __grid_constant__ Table<CAP> tab, const NormArgs a) {
  __shared__ float s_red[kWarps];
  __shared__ double s_tot[kWarps];
  __shared__ bool s_last;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float sum = 0.f;
  int at = 0;
  int64_t end = 0;
  for (int64_t chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    if (chunk >= end) {
      at = tensor_of(tab, a.n, chunk);
      end = at + 1 < a.n ? tab.t[at + 1].chunk0 : a.chunks;
    }
    const Tensor& x = tab.t[at];
    const int64_t e0 = (chunk - x.chunk0) * kNormChunk, rest = x.n - e0;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (x.vec && rest >= kNormChunk) {  // all loads of the chunk in flight
      if (!x.g_bf16) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x.g) + e0) + threadIdx.x;
        float4 v[kNormChunk / (kThreads * 4)];
#pragma unroll
        for (int q = 0; q < kNormChunk / (kThreads * 4); ++q) v[q] = __ldcs(p + q * kThreads);
#pragma unroll
        for (int q = 0; q < kNormChunk / (kThreads * 4); ++q) {
          s[0] = fmaf(v[q].x, v[q].x, s[0]); s[1] = fmaf(v[q].y, v[q].y, s[1]);
          s[2] = fmaf(v[q].z, v[q].z, s[2]); s[3] = fmaf(v[q].w, v[q].w, s[3]);
        }
      } else {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x.g) + e0) + threadIdx.x;
        uint4 v[kNormChunk / (kThreads * 8)];
#pragma unroll
        for (int q = 0; q < kNormChunk / (kThreads * 8); ++q) v[q] = __ldcs(p + q * kThreads);
#pragma unroll
        for (int q = 0; q < kNormChunk / (kThreads * 8); ++q) {
          const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]));
            s[k] = fmaf(f.x, f.x, s[k]);
            s[k] = fmaf(f.y, f.y, s[k]);
          }
        }
      }
    } else {
      const int n = int(min(int64_t(kNormChunk), rest));
      auto add = [&](const auto* p) {
        for (int q0 = threadIdx.x; q0 < n; q0 += 8 * kThreads) {
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = q0 + q * kThreads < n ? to_f32(p[q0 + q * kThreads]) : 0.f;
#pragma unroll
          for (int q = 0; q < 8; ++q) s[q & 3] = fmaf(v[q], v[q], s[q & 3]);
        }
      };
      if (x.g_bf16) add(static_cast<const __nv_bfloat16*>(x.g) + e0);
      else add(static_cast<const float*>(x.g) + e0);
    }
    sum += (s[0] + s[1]) + (s[2] + s[3]);
  }
  sum = block_sum_all<kWarps>(sum, s_red);
  double d = 0.0;
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) {
      a.part[blockIdx.x] = sum;
      __threadfence();
      s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    for (int i = threadIdx.x; i < int(gridDim.x); i += kThreads) d += double(__ldcg(a.part + i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (lane == 0) s_tot[warp] = d;
    __syncthreads();
    d = lane < kWarps ? s_tot[lane] : 0.0;
#pragma unroll
    for (int off = kWarps / 2; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    if (threadIdx.x == 0) *a.ticket = 0u;
  } else {
    d = double(sum);
  }
  if (threadIdx.x == 0) {
    if (!a.first) d += *a.total;
    if (!a.last) *a.total = d;
    // the fp32 root where the sum is in its range (the fp64 one takes microseconds)
    else *a.out = d > 1e-30 && d < 1e30 ? __fsqrt_rn(float(d)) : float(sqrt(d));
  }
}

int check_params(const moe_param_t* t, int n, bool step) {
  if (n < 0 || (n > 0 && !t)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const moe_param_t& x = t[i];
    if (x.n < 0 || x.n > (int64_t(1) << 48)) return MOE_ERR_INVALID_ARG;
    if (x.g_dtype != MOE_F32 && x.g_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (x.n > 0 && !x.g) return MOE_ERR_INVALID_ARG;
    if (!step) continue;
    if (x.p_dtype != MOE_F32 && x.p_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (x.n > 0 && !x.p) return MOE_ERR_INVALID_ARG;
    if (x.first < 0 || x.first % kBlock != 0 || x.first > (int64_t(1) << 48)) return MOE_ERR_INVALID_ARG;
    if (!(x.weight_decay >= 0.0) || !std::isfinite(x.weight_decay)) return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

bool on(const void* p, size_t b) { return reinterpret_cast<uintptr_t>(p) % b == 0; }

constexpr int kMost = 448;  // tensors of a launch: 448 x 72 bytes of the 32 KB that arguments may have

// Fills the table from t[at ..], skipping empty tensors; returns the next index.
template <int CAP>
int fill(Table<CAP>& tab, const moe_param_t* t, int n, int at, double lr, bool step, int* used, int64_t* chunks) {
  *used = 0;
  *chunks = 0;
  for (; at < n && *used < CAP; ++at) {
    const moe_param_t& x = t[at];
    if (x.n == 0) continue;
    Tensor& d = tab.t[(*used)++];
    d.p = step ? x.p : nullptr;
    d.g = x.g;
    d.copy = step ? x.copy : nullptr;
    d.n = x.n;
    d.first = step ? x.first : 0;
    d.chunk0 = *chunks;
    d.wd = step ? float(x.weight_decay) : 0.f;
    d.decay = step ? float(1.0 - lr * x.weight_decay) : 1.f;
    d.p_bf16 = step && x.p_dtype == MOE_BF16;
    d.g_bf16 = x.g_dtype == MOE_BF16;
    d.vec = on(x.g, d.g_bf16 && step ? 8 : 16) && (!step || (on(x.p, d.p_bf16 ? 8 : 16) && on(x.copy, 8)));
    const int64_t chunk = step ? kChunk : kNormChunk;
    *chunks += (x.n + chunk - 1) / chunk;
  }
  return at;
}

// f(table, used, chunks, last) for each launch's tensors, in the smallest table that takes them all
template <int CAP, typename F>
int launches(const moe_param_t* t, int n, double lr, bool step, F&& f) {
  Table<CAP> tab;
  int at = 0;
  do {
    int used;
    int64_t chunks;
    const int next = fill(tab, t, n, at, lr, step, &used, &chunks);
    bool last = true;  // nothing but empty tensors follows
    for (int i = next; i < n && last; ++i) last = t[i].n == 0;
    const int rc = f(tab, used, chunks, at == 0, last);
    if (rc != MOE_OK || last) return rc;
    at = next;
  } while (at < n);
  return MOE_OK;
}
template <typename F>
int with_table(const moe_param_t* t, int n, double lr, bool step, F&& f) {
  if (n <= 16) return launches<16>(t, n, lr, step, f);
  if (n <= 96) return launches<96>(t, n, lr, step, f);
  return launches<kMost>(t, n, lr, step, f);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_adamw_step(const moe_adamw_t* a, const moe_param_t* params, int n, void* m, void* v, float* m_scale,
                   float* v_scale, double* clock, const float* lr, const float* norm, void* ws, size_t ws_bytes,
                   moe_stream_t stream) {
  if (!a || (a->bits != 32 && a->bits != 8)) return MOE_ERR_INVALID_ARG;
  if (!(a->beta1 >= 0.0 && a->beta1 < 1.0) || !(a->beta2 >= 0.0 && a->beta2 < 1.0) || !(a->eps >= 0.f) ||
      !std::isfinite(a->eps) || !std::isfinite(a->lr))
    return MOE_ERR_INVALID_ARG;
  if (norm && !(a->max_norm > 0.f)) return MOE_ERR_INVALID_ARG;
  const int rc = check_params(params, n, true);
  if (rc != MOE_OK) return rc;
  if (!clock || !on(clock, 8)) return MOE_ERR_INVALID_ARG;
  bool any = false;
  for (int i = 0; i < n && !any; ++i) any = params[i].n > 0;
  if (any && (!m || !v || !on(m, 16) || !on(v, 16))) return MOE_ERR_INVALID_ARG;
  if (any && a->bits == 8 && (!m_scale || !v_scale)) return MOE_ERR_INVALID_ARG;
  if (!ws || !on(ws, 256) || ws_bytes < 256) return MOE_ERR_WORKSPACE;
  StepArgs s;
  s.m = m; s.v = v; s.m_scale = m_scale; s.v_scale = v_scale;
  s.clock = clock; s.lr_dev = lr; s.norm = norm;
  s.ticket = static_cast<unsigned*>(ws) + 1;
  s.beta1 = a->beta1; s.beta2 = a->beta2;
  s.lr = float(a->lr);
  s.b1 = float(a->beta1); s.c1 = float(1.0 - a->beta1);
  s.b2 = float(a->beta2); s.c2 = float(1.0 - a->beta2);
  s.eps = a->eps; s.max_norm = a->max_norm;
  s.seed = a->bits == 8 ? a->seed : -1;
  return with_table(params, n, a->lr, true, [&](const auto& tab, int used, int64_t chunks, bool, bool last) {
    constexpr int CAP = sizeof(tab.t) / sizeof(Tensor);
    s.n = used; s.chunks = chunks; s.last = last;
    const unsigned grid = unsigned(std::max<int64_t>(1, std::min<int64_t>(chunks, 4 * num_sms())));
    auto kern = a->bits == 8 ? adamw_kernel<8, CAP> : adamw_kernel<32, CAP>;
    return launch_kernel(kern, dim3(grid), dim3(kThreads), 0, stream, tab, s);
  });
}

int moe_adamw_values(const void* m, const void* v, const float* m_scale, const float* v_scale, int64_t n, float* m_out,
                     float* v_out, moe_stream_t stream) {
  if (n < 0 || n % kBlock != 0) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!m || !v || !m_scale || !v_scale || !m_out || !v_out) return MOE_ERR_INVALID_ARG;
  if (!on(m, 4) || !on(v, 4) || !on(m_out, 16) || !on(v_out, 16)) return MOE_ERR_INVALID_ARG;
  const unsigned grid = unsigned(std::min<int64_t>((n / 4 + kThreads - 1) / kThreads, 16 * num_sms()));
  return launch_kernel(adamw_values_kernel, dim3(grid), dim3(kThreads), 0, stream, static_cast<const int8_t*>(m),
                       static_cast<const uint8_t*>(v), m_scale, v_scale, n, m_out, v_out);
}

int moe_grad_norm_workspace_bytes(size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = 256 + kNormSlots * sizeof(float);
  return MOE_OK;
}

int moe_grad_norm(const moe_param_t* params, int n, float* out, void* ws, size_t ws_bytes, moe_stream_t stream) {
  const int rc = check_params(params, n, false);
  if (rc != MOE_OK) return rc;
  if (!out) return MOE_ERR_INVALID_ARG;
  size_t need;
  moe_grad_norm_workspace_bytes(&need);
  if (!ws || !on(ws, 256) || ws_bytes < need) return MOE_ERR_WORKSPACE;
  NormArgs a;
  a.out = out;
  a.ticket = static_cast<unsigned*>(ws) + 1;
  a.total = reinterpret_cast<double*>(static_cast<char*>(ws) + 64);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + 256);
  return with_table(params, n, 0.0, false, [&](const auto& tab, int used, int64_t chunks, bool first, bool last) {
    constexpr int CAP = sizeof(tab.t) / sizeof(Tensor);
    a.n = used; a.chunks = chunks; a.first = first; a.last = last;
    const int64_t most = std::min<int64_t>(kNormSlots, 4 * num_sms());
    const unsigned grid = unsigned(std::max<int64_t>(1, std::min(chunks, most)));
    return launch_kernel(grad_norm_kernel<CAP>, dim3(grid), dim3(kThreads), 0, stream, tab, a);
  });
}

}  // extern "C"
