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
// full turn that pair i advances per position, in units of 2^-64: position *
// turns mod 2^64 is then the exact phase (the product's multiple of a turn
// falls off the top), where an fp32 angle has lost its last bits long before
// position 10^5.
struct RopeTable {
  uint64_t turns[kMaxRopePairs];
  float mscale;         // factor on the rotated values (1 except for YaRN)
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

// cos and sin (times mscale) of the eight pairs of chunk c at a position; sn
// is negated for the inverse rotation.  The nearest quarter turn comes off the
// top two bits of the phase, and the rest, within +-pi/4, goes into the Taylor
// polynomials: their first omitted terms are below 2e-9 (x^11/11!) and 2e-10
// (x^12/12!).  Two angles share each multiply-add.
__device__ __forceinline__ void rope_angles(const RopeTable& t, int c, int pos, bool inverse, float (&cs)[8],
                                            float (&sn)[8]) {
  const uint32_t neg = inverse ? 0x80000000u : 0u;
  const float m = t.mscale;
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    uint32_t k[2];
    float x0, x1, y0, y1, s0, s1, c0, c1;
    float r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t ph = static_cast<uint32_t>(
          (static_cast<uint64_t>(static_cast<int64_t>(pos)) * t.turns[8 * c + e + i]) >> 32);
      k[i] = (ph + 0x20000000u) >> 30;
      r[i] = static_cast<float>(static_cast<int32_t>(ph - (k[i] << 30)));
    }
    fmul2v(x0, x1, r[0], r[1], 1.46291807926715968e-9f, 1.46291807926715968e-9f);  // 2 pi / 2^32
    fmul2v(y0, y1, x0, x1, x0, x1);
    ffma2(s0, s1, y0, y1, 2.75573192e-6f, -1.98412698e-4f);  // 1 / 9!, -1 / 7!, ...
    ffma2v(s0, s1, s0, s1, y0, y1, 8.33333333e-3f, 8.33333333e-3f);
    ffma2v(s0, s1, s0, s1, y0, y1, -1.66666667e-1f, -1.66666667e-1f);
    ffma2v(s0, s1, s0, s1, y0, y1, 1.f, 1.f);
    fmul2v(s0, s1, s0, s1, x0, x1);
    ffma2(c0, c1, y0, y1, -2.75573192e-7f, 2.48015873e-5f);
    ffma2v(c0, c1, c0, c1, y0, y1, -1.38888889e-3f, -1.38888889e-3f);
    ffma2v(c0, c1, c0, c1, y0, y1, 4.16666667e-2f, 4.16666667e-2f);
    ffma2v(c0, c1, c0, c1, y0, y1, -0.5f, -0.5f);
    ffma2v(c0, c1, c0, c1, y0, y1, 1.f, 1.f);
    fmul2v(s0, s1, s0, s1, m, m);
    fmul2v(c0, c1, c0, c1, m, m);
    const float sv[2] = {s0, s1}, cv[2] = {c0, c1};
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
// x[8..16), by cs = (cos, sin) of the first and of the second.
__device__ __forceinline__ void rope_rotate2(bool interleaved, int j, float4 cs, float (&x)[16]) {
  if (interleaved) {
    const float a0 = x[4 * j], b0 = x[4 * j + 1], a1 = x[4 * j + 2], b1 = x[4 * j + 3];
    x[4 * j] = a0 * cs.x - b0 * cs.y;
    x[4 * j + 1] = b0 * cs.x + a0 * cs.y;
    x[4 * j + 2] = a1 * cs.z - b1 * cs.w;
    x[4 * j + 3] = b1 * cs.z + a1 * cs.w;
  } else {
    const float a0 = x[2 * j], b0 = x[8 + 2 * j], a1 = x[2 * j + 1], b1 = x[9 + 2 * j];
    x[2 * j] = a0 * cs.x - b0 * cs.y;
    x[8 + 2 * j] = b0 * cs.x + a0 * cs.y;
    x[2 * j + 1] = a1 * cs.z - b1 * cs.w;
    x[9 + 2 * j] = b1 * cs.z + a1 * cs.w;
  }
}
__device__ __forceinline__ void rope_rotate(bool interleaved, const float (&cs)[8], const float (&sn)[8],
                                            float (&x)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    rope_rotate2(interleaved, j, make_float4(cs[2 * j], sn[2 * j], cs[2 * j + 1], sn[2 * j + 1]), x);
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
