// Rotary positions on the device: the frequency table as it travels to the
// kernels, the angle of a pair at a position, and the 16-value chunks that a
// thread rotates.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "msa_internal.h"
#include "ptx.cuh"

namespace msa {

constexpr int kMaxRopePairs = 128;

// Passed by value: the kernels read it from the constant bank, so a handle
// owns no device memory and serves any device.  turns[i] is the fraction of a
// full turn that pair i advances per position, in units of 2^-64, to the
// nearest: position * turns mod 2^64 is then the phase (the product's multiple
// of a turn falls off the top) to 2^-34 of a turn at any int32 position, where
// an fp32 angle has lost its last bits long before position 10^5.
struct RopeTable {
  uint64_t turns[kMaxRopePairs];
  float mscale;         // factor on the rotated values (1 except for YaRN), and what
  float mscale_lo;      // fp32 leaves of it
  int32_t rot;          // rotated dims of a head; 0: no rotation
  int32_t interleaved;  // pairs (2i, 2i + 1); otherwise (i, i + rot / 2)
};

}  // namespace msa

struct msa_rope_s {
  msa::RopeTable table;
};

namespace msa {

#ifdef __CUDACC__

// Where thread-chunk c (16 values of a head) lies: two runs of 8 values.  A
// rotated chunk of the half layout takes the same 8 pairs from both halves;
// every other chunk is 16 consecutive values.
struct RopeChunk {
  int lo, hi;
  bool rotated;
};
__device__ __forceinline__ RopeChunk rope_chunk(const RopeTable& t, int c) {
  const bool rotated = 16 * c < t.rot;
  if (rotated && !t.interleaved) return {8 * c, t.rot / 2 + 8 * c, true};
  return {16 * c, 16 * c + 8, rotated};
}

// Two fp32 values that go through packed arithmetic together.
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  ffma2v(d.x, d.y, a.x, a.y, b.x, b.y, c.x, c.y);
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, float b, F2 c) { return fma2(a, F2{b, b}, c); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  fmul2v(d.x, d.y, a.x, a.y, b.x, b.y);
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, float b) { return mul2(a, F2{b, b}); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  fadd2v(d.x, d.y, a.x, a.y, b.x, b.y);
  return d;
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b) { return fma2(b, -1.f, a); }

// cos and sin of two angles x + xl within +-pi/4, by Taylor polynomials whose
// first omitted terms are below 2e-9 and 2e-10.
__device__ __forceinline__ void sincos_short(F2 x, F2& s, F2& co) {
  const F2 y = mul2(x, x);
  F2 p = fma2(y, 2.75573192e-6f, F2{-1.98412698e-4f, -1.98412698e-4f});  // 1/9!, -1/7!, 1/5!, -1/3!
  p = fma2(p, y, F2{8.33333333e-3f, 8.33333333e-3f});
  p = fma2(p, y, F2{-1.66666667e-1f, -1.66666667e-1f});
  s = mul2(fma2(p, y, F2{1.f, 1.f}), x);
  F2 q = fma2(y, -2.75573192e-7f, F2{2.48015873e-5f, 2.48015873e-5f});  // -1/10!, 1/8!, -1/6!, 1/4!, -1/2!
  q = fma2(q, y, F2{-1.38888889e-3f, -1.38888889e-3f});
  q = fma2(q, y, F2{4.16666667e-2f, 4.16666667e-2f});
  q = fma2(q, y, F2{-0.5f, -0.5f});
  co = fma2(q, y, F2{1.f, 1.f});
}

// The same, the nearest fp32 in all but 1 case of 200 (co) and 1 of 40 (s): only
// terms below 1/12 are rounded before the last addition.  s_lo, co_lo: what the
// two leave.
__device__ __forceinline__ void sincos_nearest(F2 x, F2 xl, F2& s, F2& s_lo, F2& co, F2& co_lo) {
  constexpr float c3 = -0x1.555556p-3f, c3l = 0x1.555556p-28f;  // -1/3!
  const F2 zero{0.f, 0.f}, one{1.f, 1.f};
  // y + yl = x^2, z + zl = x^3
  const F2 y = mul2(x, x), half = mul2(y, -0.5f);
  const F2 yl = fma2(add2(x, x), xl, fma2(x, x, sub2(zero, y)));
  const F2 z = mul2(x, y);
  const F2 zl = fma2(x, yl, fma2(x, y, sub2(zero, z)));
  F2 p = fma2(y, 2.75573192e-6f, F2{-1.98412698e-4f, -1.98412698e-4f});
  p = mul2(fma2(p, y, F2{8.33333333e-3f, 8.33333333e-3f}), y);
  const F2 rest = fma2(z, c3, fma2(half, xl, fma2(z, c3l, fma2(zl, c3, fma2(z, p, xl)))));
  s = add2(x, rest);
  s_lo = sub2(rest, sub2(s, x));
  F2 q = fma2(y, -2.75573192e-7f, F2{2.48015873e-5f, 2.48015873e-5f});
  q = fma2(q, y, F2{-1.38888889e-3f, -1.38888889e-3f});
  q = fma2(q, y, F2{4.16666667e-2f, 4.16666667e-2f});
  const F2 c0 = add2(half, one);
  const F2 cl = add2(fma2(mul2(y, y), q, mul2(yl, -0.5f)), add2(half, sub2(one, c0)));
  co = add2(c0, cl);
  co_lo = sub2(cl, sub2(co, c0));
}

// cos and sin, times mscale, of the eight pairs of chunk c at a position; sn is
// negated for the inverse rotation.  The nearest quarter turn comes off the top
// two bits of the phase, the rest is within +-pi/4.
//
// kNearest: rounded as cosines computed in fp64 are, so that a rotation from
// here has the bits of an elementwise one, and a cache quantised by either holds
// the same codes.
template <bool kNearest = true>
__device__ __forceinline__ void rope_angles(const RopeTable& t, int c, int pos, bool inverse, float (&cs)[8],
                                            float (&sn)[8]) {
  constexpr float k1 = 0x1.921fb6p-30f, k2 = -0x1.777a5cp-55f;  // 2 pi / 2^32
  const uint32_t neg = inverse ? 0x80000000u : 0u;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    uint32_t k[2];
    float hi[2], lo[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * t.turns[8 * c + e + i];
      const uint32_t ph = static_cast<uint32_t>(phase >> 32);
      k[i] = (ph + 0x20000000u) >> 30;
      const int r = static_cast<int>(ph - (k[i] << 30));  // 30 bits
      hi[i] = static_cast<float>(kNearest ? r & ~0xFF : r);  // the top 22 are exact
      lo[i] = kNearest ? fmaf(static_cast<float>(static_cast<uint32_t>(phase)), 0x1p-32f,
                              static_cast<float>(r & 0xFF))
                       : 0.f;
    }
    const F2 rh{hi[0], hi[1]}, rl{lo[0], lo[1]}, zero{0.f, 0.f};
    const F2 x0 = mul2(rh, k1);
    F2 s, co;
    if (kNearest) {
      F2 xl = fma2(rl, k1, fma2(rh, k2, fma2(rh, k1, sub2(zero, x0)))), sl, cl;
      const F2 x = add2(x0, xl);
      sincos_nearest(x, sub2(xl, sub2(x, x0)), s, sl, co, cl);
      if (t.mscale != 1.f) {
        const F2 sm = mul2(s, t.mscale), cm = mul2(co, t.mscale);
        s = add2(sm, fma2(s, t.mscale_lo, fma2(sl, t.mscale, fma2(s, t.mscale, sub2(zero, sm)))));
        co = add2(cm, fma2(co, t.mscale_lo, fma2(cl, t.mscale, fma2(co, t.mscale, sub2(zero, cm)))));
      }
    } else {
      sincos_short(x0, s, co);
      s = mul2(s, t.mscale);
      co = mul2(co, t.mscale);
    }
    const float sv[2] = {s.x, s.y}, cv[2] = {co.x, co.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = __float_as_uint(sv[i]), b = __float_as_uint(cv[i]);
      const bool odd = k[i] & 1u;
      sn[e + i] = __uint_as_float((odd ? b : a) ^ ((k[i] & 2u) << 30) ^ neg);
      cs[e + i] = __uint_as_float((odd ? a : b) ^ (((k[i] + 1u) & 2u) << 30));
    }
  }
}

// Rotates pairs 2 j and 2 j + 1 of a chunk, whose two runs are x[0..8) and
// x[8..16), by cs = (cos, cos, sin, sin) of the two: products rounded, then
// their sums, as elementwise arithmetic does it.
__device__ __forceinline__ void rope_rotate2(bool interleaved, int j, float4 cs, float (&x)[16]) {
  // (the sums are scalar: a packed product and a packed sum may become one
  // multiply-add, whose product is not rounded)
  auto turn = [&](float& a0, float& b0, float& a1, float& b1) {
    const F2 a{a0, a1}, b{b0, b1}, c{cs.x, cs.y}, s{cs.z, cs.w};
    const F2 ac = mul2(a, c), bs = mul2(b, s), bc = mul2(b, c), as = mul2(a, s);
    a0 = __fsub_rn(ac.x, bs.x), a1 = __fsub_rn(ac.y, bs.y);
    b0 = __fadd_rn(bc.x, as.x), b1 = __fadd_rn(bc.y, as.y);
  };
  if (interleaved)
    turn(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
  else
    turn(x[2 * j], x[8 + 2 * j], x[2 * j + 1], x[9 + 2 * j]);
}
__device__ __forceinline__ void rope_rotate(bool interleaved, const float (&cs)[8], const float (&sn)[8],
                                            float (&x)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    rope_rotate2(interleaved, j, make_float4(cs[2 * j], cs[2 * j + 1], sn[2 * j], sn[2 * j + 1]), x);
}

__device__ __forceinline__ void unpack8(uint4 v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  unpack8(*reinterpret_cast<const uint4*>(p), x);
}
__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]),
                                            bf16x2_bits(x[4], x[5]), bf16x2_bits(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// A chunk's two runs of 8 values as they come from memory.
template <typename T>
struct Raw16;
template <>
struct Raw16<__nv_bfloat16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* lo, const __nv_bfloat16* hi) {
    a = *reinterpret_cast<const uint4*>(lo);
    b = *reinterpret_cast<const uint4*>(hi);
  }
  __device__ __forceinline__ void unpack(float (&x)[16]) const {
    unpack8(a, x);
    unpack8(b, x + 8);
  }
};
template <>
struct Raw16<float> {
  float v[16];
  __device__ __forceinline__ void load(const float* lo, const float* hi) {
    load8(lo, v);
    load8(hi, v + 8);
  }
  __device__ __forceinline__ void unpack(float (&x)[16]) const {
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = v[e];
  }
};

#endif  // __CUDACC__

}  // namespace msa
