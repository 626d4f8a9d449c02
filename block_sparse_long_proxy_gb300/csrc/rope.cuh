// Rotary positions on the device: the frequency table as it travels to the
// kernels, the angle of a pair at a position, and the 16-value chunks that a
// thread rotates.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "msa_internal.h"

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
// is negated for the inverse rotation.  The top 32 bits of the phase as a
// signed number are the angle in units of 2^-31 half turns.
__device__ __forceinline__ void rope_angles(const RopeTable& t, int c, int pos, bool inverse, float (&cs)[8],
                                            float (&sn)[8]) {
  const float a = t.mscale, b = inverse ? -t.mscale : t.mscale;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * t.turns[8 * c + e];
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &sn[e], &cs[e]);
    cs[e] *= a;
    sn[e] *= b;
  }
}

// x[0..8) and x[8..16) are a chunk's two runs
__device__ __forceinline__ void rope_rotate(bool interleaved, const float (&cs)[8], const float (&sn)[8],
                                            float (&x)[16]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (interleaved) {
      const float p = x[2 * e], q = x[2 * e + 1];
      x[2 * e] = p * cs[e] - q * sn[e];
      x[2 * e + 1] = q * cs[e] + p * sn[e];
    } else {
      const float p = x[e], q = x[8 + e];
      x[e] = p * cs[e] - q * sn[e];
      x[8 + e] = q * cs[e] + p * sn[e];
    }
  }
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
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

#endif  // __CUDACC__

}  // namespace msa
