// The writers of the paged caches: a batch's new K, V and proxy K rows,
// rotated and quantised, to their pages and slots; and the backward, which
// takes the gradient pages back to rows.
//
// The unit of work is one page that gets rows, from the plan's table: its
// rows first_row .. first_row + n go to slots slot0 .. slot0 + n of the page.
// A page is touched by one unit of a call, so nothing is summed or written
// twice, and a scale shared by a whole page is known to the CTA that has all
// of the page's new rows in registers.
//
// e4m3 with a scale for each (page, KV head):  s = 2^e, e the least integer
// with amax <= 448 * 2^e.  A power of two costs e4m3 nothing (it is a
// floating-point format; x / s is exact) and makes the page's codes nearly
// independent of how its rows came in: where a later row raises the scale,
// the old codes are multiplied by a power of two, which changes no bits
// except those that fall below e4m3's smallest step.
#include <cuda_fp16.h>

#include <algorithm>

#include "ptx.cuh"
#include "rope.cuh"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kKvThreads = 512;
constexpr int kPkThreads = 128;
constexpr int kMinExp = -40, kMaxExp = 40;

struct AppendUnit {
  int32_t entry;    // index in kv_indices
  int32_t row;      // first new row
  int32_t pos;      // its key position in the sequence
  int32_t slot0_n;  // its slot, and the number of rows << 8
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {  // saturating; NaN stays NaN
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}
__device__ __forceinline__ uint2 e4m3x8(const float* x) {
  return make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// least e in [kMinExp, kMaxExp] with amax <= 448 * 2^e; amax >= 0 and finite
__device__ __forceinline__ int block_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
  return min(max(e, kMinExp), kMaxExp);
}

// x0 / s and x1 / s to nearest, given the nearest reciprocal of s: one residual
// step on x * inv (Markstein 1990).  Quotients that saturate, infinities and NaN
// are left as the product has them.
__device__ __forceinline__ void quotient2(float& x0, float& x1, float s, float inv) {
  const F2 x{x0, x1}, q = mul2(x, inv), r = fma2(fma2(q, -s, x), inv, q);
  x0 = fabsf(q.x) < 512.f ? r.x : q.x;
  x1 = fabsf(q.y) < 512.f ? r.y : q.y;
}

// Sixteen consecutive values as their even ones and their odd ones, and back:
// interleaved pairs then rotate, and pack into bytes, as halves do.
__device__ __forceinline__ void unpack_pairs(uint4 a, uint4 b, float (&x)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = __uint_as_float(w[i] << 16);
    x[8 + i] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void pack_pairs(float (&x)[16]) {
  float y[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[2 * i] = x[i], y[2 * i + 1] = x[8 + i];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = y[i];
}

// four e4m3 codes times a factor, rounded to e4m3 again
__device__ __forceinline__ uint32_t rescale4(uint32_t v, float f) {
  const uint32_t a = e4m3x2_to_f16x2(v), b = e4m3x2_to_f16x2(v >> 16);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return e4m3x4(x.x * f, x.y * f, y.x * f, y.y * f);
}

// K (which 0, rotated) or V (1) of one page, a few KV heads.
//
// Bound by HBM for long appends.  A thread holds 16 values of one row, or of
// two, from the load through the rotation and the page's amax to the codes: the
// rows are read once.  The cos and sin of the page's rows go into shared
// memory and serve all heads of the CTA (with eight angles computed for every
// 16 values the call took 67 us, half of it issuing instructions), and the
// next head's rows are on their way while this one's amax is reduced.  32768 rows, 8 heads, d
// 128 (201 MB): 41.5 us, 4.8 TB/s (2.4 us less with the shorter angle polynomials,
// whose last bits change a few codes).
enum RopeKind { kPlain, kHalf, kInterleaved };

struct KvAppendArgs {
  const AppendUnit* units;
  const __nv_bfloat16* x[2];  // K, V
  int64_t stride[2];
  void* pages[2];
  float* scale[2];
  const int32_t* positions;
  const int32_t* kv_indices;
  int64_t num_pages;
  int32_t hkv;
  int32_t heads_per_cta[2];  // K, V
  int32_t groups[2];         // CTAs a unit that makes
  int32_t k_ctas;            // those of K come first
  uint32_t* err;
};

template <int D, msa_kv_dtype KIND, RopeKind ROPE>
__device__ __forceinline__ void kv_append(const RopeTable& tab, const KvAppendArgs& a, int which, int cta) {
  constexpr int kChunks = D / 16, kRows = kKvThreads / kChunks, kPasses = 128 / kRows;
  extern __shared__ float4 angles[];  // [row][4][kChunks]: cos, cos, sin, sin of pairs 2 j and 2 j + 1 of a chunk
  __shared__ uint32_t warp_max[2][kKvThreads / 32];
  const AppendUnit u = a.units[cta / a.groups[which]];
  const int64_t page = a.kv_indices[u.entry];
  const int slot0 = u.slot0_n & 0xFF, n = u.slot0_n >> 8;
  const int c = threadIdx.x % kChunks, r0 = threadIdx.x / kChunks;
  RopeChunk ch{16 * c, 16 * c + 8, false};
  if (ROPE != kPlain) ch = rope_chunk(tab, c);
  const int h0 = cta % a.groups[which] * a.heads_per_cta[which], h1 = min(a.hkv, h0 + a.heads_per_cta[which]);
  const __nv_bfloat16* src[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) src[p] = a.x[which] + (u.row + p * kRows + r0) * a.stride[which];
  uint4 raw[kPasses][2];
  auto load = [&](int h) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p)
      if (p * kRows + r0 < n) {
        const __nv_bfloat16* at = src[p] + h * D;
        raw[p][0] = *reinterpret_cast<const uint4*>(at + ch.lo);
        raw[p][1] = *reinterpret_cast<const uint4*>(at + ch.hi);
      }
  };
  if (ROPE == kPlain) load(h0);
  if (page < 0 || page >= a.num_pages) {
    if (threadIdx.x == 0) atomicOr(a.err, kErrDeviceCheck);
    return;
  }
  if (ROPE != kPlain && ch.rotated) {
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int i = p * kRows + r0;
      if (i < n) {
        float cs[8], sn[8];
        rope_angles(tab, c, a.positions ? a.positions[u.row + i] : u.pos + i, false, cs, sn);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          angles[(i * 4 + j) * kChunks + c] = make_float4(cs[2 * j], cs[2 * j + 1], sn[2 * j], sn[2 * j + 1]);
      }
    }
  }  // every thread reads back what it wrote
  if (ROPE != kPlain) load(h0);  // not before: the angles take the registers
  for (int h = h0; h < h1; ++h) {
    float x[kPasses][16];
    float amax = 0.f;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int i = p * kRows + r0;
      if (i < n) {
        if (ROPE == kInterleaved)
          unpack_pairs(raw[p][0], raw[p][1], x[p]);
        else
          unpack8(raw[p][0], x[p]), unpack8(raw[p][1], x[p] + 8);
        if (ROPE != kPlain && ch.rotated) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            rope_rotate2(false, j, angles[(i * 4 + j) * kChunks + c], x[p]);
        }
        if (KIND == MSA_KV_FP8_E4M3_BLOCK) {
#pragma unroll
          for (int e = 0; e < 16; e += 2) amax = fmax3(amax, fabsf(x[p][e]), fabsf(x[p][e + 1]));  // NaN is passed over
        }
      }
    }
    if (h + 1 < h1) load(h + 1);
    const int64_t head_row = (page * a.hkv + h) * 128;  // first row of the (page, head) in the pool
    if (KIND == MSA_KV_BF16) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.pages[which]) + (head_row + slot0) * D;
#pragma unroll
      for (int p = 0; p < kPasses; ++p) {
        const int i = p * kRows + r0;
        if (i < n) {
          if (ROPE == kInterleaved) pack_pairs(x[p]);
          store8(dst + i * D + ch.lo, x[p]);
          store8(dst + i * D + ch.hi, x[p] + 8);
        }
      }
      continue;
    }
    uint8_t* pool = static_cast<uint8_t*>(a.pages[which]) + head_row * D;
    float by, inv = 0.f;  // the codes are x * by (block) or x / by (one scale a head)
    if (KIND == MSA_KV_FP8_E4M3_BLOCK) {
      float* sp = a.scale[which] + page * a.hkv + h;
      const float old = slot0 > 0 ? *sp : 0.f;  // rows came before: the scale only grows
      // one barrier a head: the buffers alternate
      auto cta_max = [&](float m, int buf) {  // of values >= 0, whose bits order as they do
        const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
        if ((threadIdx.x & 31) == 0) warp_max[buf][threadIdx.x >> 5] = w;
        __syncthreads();
        return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, warp_max[buf][threadIdx.x % (kKvThreads / 32)]));
      };
      amax = cta_max(amax, h & 1);
      if (amax == INFINITY) {  // infinities saturate, they set no scale
        float fin = 0.f;
#pragma unroll
        for (int p = 0; p < kPasses; ++p)
          if (p * kRows + r0 < n)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (fabsf(x[p][e]) < INFINITY) fin = fmaxf(fin, fabsf(x[p][e]));
        __syncthreads();
        amax = cta_max(fin, h & 1);
      }
      int e = block_exp(amax);
      if (slot0 > 0) {
        if (!(old > 0.f && old <= pow2(kMaxExp))) {  // never written: the old slots keep their bytes
          if (threadIdx.x == 0) atomicOr(a.err, kErrDeviceCheck);
        } else {
          // another writer's scale need not be a power of two: round it up to one;
          // below the least it counts as that, as the attention has it
          const float was = fmaxf(old, pow2(kMinExp));
          const uint32_t ou = __float_as_uint(was);
          e = max(e, static_cast<int>(ou >> 23) - 127 + ((ou & 0x7FFFFFu) != 0u ? 1 : 0));
          const float f = was * pow2(-e);
          if (f != 1.f) {
            uint4* q = reinterpret_cast<uint4*>(pool);
            for (int i = threadIdx.x; i < slot0 * (D / 16); i += kKvThreads) {
              uint4 w = q[i];
              w.x = rescale4(w.x, f), w.y = rescale4(w.y, f), w.z = rescale4(w.z, f), w.w = rescale4(w.w, f);
              q[i] = w;
            }
          }
        }
      }
      if (threadIdx.x == 0) *sp = pow2(e);  // every thread read the old one before the barrier
      by = pow2(-e);
    } else {
      by = a.scale[which][h];
      inv = __frcp_rn(by);
    }
    uint8_t* dst = pool + slot0 * D;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int i = p * kRows + r0;
      if (i < n) {
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          if (KIND == MSA_KV_FP8_E4M3_BLOCK)
            fmul2v(x[p][e], x[p][e + 1], x[p][e], x[p][e + 1], by, by);
          else
            quotient2(x[p][e], x[p][e + 1], by, inv);
        }
        if (ROPE == kInterleaved) pack_pairs(x[p]);
        *reinterpret_cast<uint2*>(dst + i * D + ch.lo) = e4m3x8(x[p]);
        *reinterpret_cast<uint2*>(dst + i * D + ch.hi) = e4m3x8(x[p] + 8);
      }
    }
  }
}

template <int D, msa_kv_dtype KIND>
__global__ void __launch_bounds__(kKvThreads, 2)
    kv_append_kernel(const __grid_constant__ RopeTable tab, const __grid_constant__ KvAppendArgs a) {
  pdl_wait();
  // one body for each way of rotating: what differs is which values pair up
  const int which = static_cast<int>(blockIdx.x) >= a.k_ctas, cta = blockIdx.x - which * a.k_ctas;
  if (which == 1 || tab.rot == 0)
    kv_append<D, KIND, kPlain>(tab, a, which, cta);
  else if (tab.interleaved)
    kv_append<D, KIND, kInterleaved>(tab, a, 0, cta);
  else
    kv_append<D, KIND, kHalf>(tab, a, 0, cta);
}

// Proxy K rows of one page, to any of three pools.
//
// NVFP4: block scale bs = e4m3(amax16 / (6 g)), codes e2m1(x / (bs g)), both
// to nearest with ties to even.  bf16 keys over a scale measured on bf16 data
// fall on and next to the borders between codes, where a rounded quotient
// takes the wrong side; so both roundings compare x with border * bs * g by
// one fused multiply-add, whose sign is exact (border * bs has at most 8 bits).
struct ProxyPools {
  __nv_bfloat16* bf16;
  uint8_t* e4m3;
  const float* e4m3_scale;
  uint8_t* codes;
  uint8_t* block_scales;
  const float* global_scale;
};

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  const uint32_t h = e4m3x2_to_f16x2(code);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

// the e4m3 code nearest to amax / (6 g)
__device__ __forceinline__ uint32_t nvfp4_block_scale(float amax, float g) {
  uint32_t c = e4m3x2(__fdiv_rn(amax, 6.f * g), 0.f) & 0xFFu;
  if (c >= 0x7Fu) return c;  // NaN keys
  // the quotient is off by at most an ulp: check both borders of the code
  const float v = e4m3_value(c);
  if (c < 0x7Eu) {
    const float d = fmaf(-3.f * (v + e4m3_value(c + 1)), g, amax);  // amax - 6 g (v + next) / 2
    if (d > 0.f || (d == 0.f && (c & 1u))) return c + 1;
  }
  if (c > 0) {
    const float d = fmaf(-3.f * (v + e4m3_value(c - 1)), g, amax);
    if (d < 0.f || (d == 0.f && (c & 1u))) return c - 1;
  }
  return c;
}

// the e2m1 code nearest to x / (bs g); bs > 0
__device__ __forceinline__ uint32_t nvfp4_code(float x, float bs, float g) {
  const float a = fabsf(x);
  uint32_t c = 0;
  c += fmaf(-0.25f * bs, g, a) > 0.f;
  c += fmaf(-0.75f * bs, g, a) >= 0.f;
  c += fmaf(-1.25f * bs, g, a) > 0.f;
  c += fmaf(-1.75f * bs, g, a) >= 0.f;
  c += fmaf(-2.5f * bs, g, a) > 0.f;
  c += fmaf(-3.5f * bs, g, a) >= 0.f;
  c += fmaf(-5.f * bs, g, a) > 0.f;
  return c | (__float_as_uint(x) >> 31 << 3);
}

//
// Rows share nothing, so blockIdx.y takes a page's rows by kRows: a thread has
// 16 values of one row.  13,000 rows of 64 (6.7 MB) to bf16 and NVFP4: 5.2 us
// (7.8 with a CTA a page), a few dependent reads and the launch.
template <int DP>
__global__ void __launch_bounds__(kPkThreads)
    pk_append_kernel(const __grid_constant__ RopeTable tab, const AppendUnit* __restrict__ units,
                     const __nv_bfloat16* __restrict__ pk, int64_t stride, const int32_t* __restrict__ positions,
                     const int32_t* __restrict__ kv_indices, int64_t num_pages,
                     const __grid_constant__ ProxyPools pools, uint32_t* err) {
  pdl_wait();
  constexpr int kChunks = DP / 16, kRows = kPkThreads / kChunks;
  __shared__ __align__(16) float rows[kRows][DP];  // rotated: NVFP4 blocks are 16 consecutive dims
  const AppendUnit u = units[blockIdx.x];
  const int64_t page = kv_indices[u.entry];
  const int slot0 = u.slot0_n & 0xFF, n = u.slot0_n >> 8;
  const int c = threadIdx.x % kChunks, r = threadIdx.x / kChunks, i = blockIdx.y * kRows + r;
  const RopeChunk ch = rope_chunk(tab, c);
  float x[16];
  if (i < n) {
    const __nv_bfloat16* src = pk + (u.row + i) * stride;
    load8(src + ch.lo, x);
    load8(src + ch.hi, x + 8);
    if (ch.rotated) {
      float cs[8], sn[8];
      rope_angles(tab, c, positions ? positions[u.row + i] : u.pos + i, false, cs, sn);
      rope_rotate(tab.interleaved != 0, cs, sn, x);
    }
  }
  if (page < 0 || page >= num_pages) {
    if (threadIdx.x == 0) atomicOr(err, kErrDeviceCheck);
    return;
  }
  const int64_t row = page * 128 + slot0 + i;
  if (i < n) {
    if (pools.bf16) {
      store8(pools.bf16 + row * DP + ch.lo, x);
      store8(pools.bf16 + row * DP + ch.hi, x + 8);
    }
    if (pools.codes) {
      store8(&rows[r][ch.lo], x);
      store8(&rows[r][ch.hi], x + 8);
    }
    if (pools.e4m3) {
      const float scale = *pools.e4m3_scale, inv = __frcp_rn(scale);
#pragma unroll
      for (int e = 0; e < 16; e += 2) quotient2(x[e], x[e + 1], scale, inv);
      *reinterpret_cast<uint2*>(pools.e4m3 + row * DP + ch.lo) = e4m3x8(x);
      *reinterpret_cast<uint2*>(pools.e4m3 + row * DP + ch.hi) = e4m3x8(x + 8);
    }
  }
  if (!pools.codes) return;
  __syncthreads();
  if (i >= n) return;
  load8(&rows[r][16 * c], x);
  load8(&rows[r][16 * c + 8], x + 8);
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
  const float g = *pools.global_scale;
  const uint32_t sc = nvfp4_block_scale(amax, g);
  const float bs = e4m3_value(sc);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e >> 3] |= (bs > 0.f ? nvfp4_code(x[e], bs, g) : 0u) << (4 * (e & 7));
  *reinterpret_cast<uint2*>(pools.codes + row * (DP / 2) + 8 * c) = make_uint2(w[0], w[1]);
  pools.block_scales[row * kChunks + c] = static_cast<uint8_t>(sc);
}

// Gradient pages to rows: dK (rotated back), dV and dpk (rotated back).
// blockIdx.y: KV heads of K, then of V, then the proxy head.
//
// Bound by HBM: 65536 rows, 8 heads of 128, dpk of 64 (1.1 GB) take 167 us, 6.6
// TB/s.  Each CTA computes its own angles, by the shorter polynomials, as
// nothing is quantised here; sharing them between heads, as the appends do,
// costs the occupancy that keeps the loads coming (180-190 us).
struct GradSet {
  const float* pages;
  float* rows;
  int32_t heads, d;
};

__global__ void __launch_bounds__(kThreads)
    append_bwd_kernel(const __grid_constant__ RopeTable k_tab, const __grid_constant__ RopeTable pk_tab,
                      const AppendUnit* __restrict__ units, const int32_t* __restrict__ positions,
                      const int32_t* __restrict__ kv_indices, int64_t num_pages,
                      const __grid_constant__ GradSet dk, const __grid_constant__ GradSet dv,
                      const __grid_constant__ GradSet dpk, uint32_t* err) {
  pdl_wait();
  const AppendUnit u = units[blockIdx.x];
  int h = blockIdx.y;
  int which = 0;
  if (h >= dk.heads) h -= dk.heads, which = 1;
  if (which == 1 && h >= dv.heads) h -= dv.heads, which = 2;
  const GradSet& gs = which == 0 ? dk : which == 1 ? dv : dpk;
  const RopeTable& tab = which == 2 ? pk_tab : k_tab;
  const int64_t page = kv_indices[u.entry];
  const bool ok = page >= 0 && page < num_pages;  // a page outside the pool gives zero rows
  if (!ok && threadIdx.x == 0) atomicOr(err, kErrDeviceCheck);
  const int slot0 = u.slot0_n & 0xFF, n = u.slot0_n >> 8;
  const int chunks = gs.d / 16, rows = kThreads / chunks;
  const int c = threadIdx.x % chunks, r = threadIdx.x / chunks;
  RopeChunk ch = rope_chunk(tab, c);
  if (which == 1) ch = {16 * c, 16 * c + 8, false};
  for (int i = r; i < n; i += rows) {
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.f;
    if (ok) {
      const float* src = gs.pages + ((page * gs.heads + h) * 128 + slot0 + i) * gs.d;
      load8(src + ch.lo, x);
      load8(src + ch.hi, x + 8);
    }
    if (ch.rotated) {
      float cs[8], sn[8];
      rope_angles<false>(tab, c, positions ? positions[u.row + i] : u.pos + i, true, cs, sn);
      rope_rotate(tab.interleaved != 0, cs, sn, x);
    }
    float* dst = gs.rows + (static_cast<int64_t>(u.row + i) * gs.heads + h) * gs.d;
    store8(dst + ch.lo, x);
    store8(dst + ch.hi, x + 8);
  }
}

const RopeTable& table_of(msa_rope_t r) {
  static const RopeTable none{};  // rot 0: nothing is rotated
  return r ? r->table : none;
}

// What every call here checks of its plan and rope.
msa_status check_append(const char* fn, msa_plan_t plan, msa_rope_t rope, int32_t d) {
  const msa_status s = check_device(fn, plan);
  if (s != MSA_OK) return s;
  if (rope && rope->table.rot > d)
    return set_error(MSA_ERR_INVALID_ARG, "%s: rotary_dim %d above the head's %d", fn, rope->table.rot, d);
  return MSA_OK;
}

msa_status check_rows(const char* fn, const char* name, const void* x, int64_t stride, int64_t width) {
  if (stride < width || stride > (int64_t(1) << 40))
    return set_error(MSA_ERR_INVALID_ARG, "%s: the row stride of %s must be at least %lld", fn, name,
                     static_cast<long long>(width));
  if (!aligned16(x) || stride % 8 != 0)
    return set_error(MSA_ERR_INVALID_ARG, "%s: rows of %s must start on 16-byte boundaries", fn, name);
  return MSA_OK;
}

template <int D, msa_kv_dtype KIND>
cudaError_t launch_kv(const msa_plan_s* p, const RopeTable& tab, KvAppendArgs a, cudaStream_t st) {
  // heads a CTA: the angles are shared while three CTAs are left for an SM
  // (32768 rows, 8 heads, d 128, shorter angles: 4 heads a CTA 42.7 us, 8 40.2)
  int hpc = 1;
  while (hpc < 8 && int64_t(p->n_append_units) * ((p->hkv + 2 * hpc - 1) / (2 * hpc)) * 2 >= 3 * p->num_sms) hpc *= 2;
  // V has no angles: smaller CTAs behind those of K fill the last round (8 heads a
  // CTA for both 43.2 us, 4 for V 41.7, 2 41.7, 1 44.3; bf16 53.1, 49.3, 49.9, 50.6)
  const int hpv = std::max(1, hpc / 2);
  a.heads_per_cta[0] = hpc, a.heads_per_cta[1] = hpv;
  a.groups[0] = (p->hkv + hpc - 1) / hpc, a.groups[1] = (p->hkv + hpv - 1) / hpv;
  const int64_t ctas = int64_t(p->n_append_units) * (a.groups[0] + a.groups[1]);
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  a.k_ctas = p->n_append_units * a.groups[0];
  auto kern = kv_append_kernel<D, KIND>;
  constexpr int kRowBytes = D * 4;  // (cos, sin) of D / 2 pairs of a row
  const int smem = (p->decode ? 1 : 128) * kRowBytes;
  // the limit is the function's, for every host thread: always the most of any plan
  if (const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * kRowBytes))
    return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kKvThreads), smem, st, tab, a);
}

}  // namespace

void append_plan_tables(msa_plan_s* p, std::vector<int32_t>& aux) {
  p->append_units_off = static_cast<int64_t>(aux.size());
  int64_t row = 0, base = 0;
  for (int s = 0; s < p->batch; ++s) {
    const int64_t kl = p->kv_lens[s];
    for (int64_t pos = kl - p->qo_lens[s]; pos < kl;) {
      const int64_t n = std::min<int64_t>(kl - pos, kPage - pos % kPage);
      const AppendUnit u{static_cast<int32_t>(base + pos / kPage), static_cast<int32_t>(row),
                         static_cast<int32_t>(pos), static_cast<int32_t>((pos % kPage) | (n << 8))};
      const int32_t* raw = reinterpret_cast<const int32_t*>(&u);
      aux.insert(aux.end(), raw, raw + sizeof(u) / 4);
      ++p->n_append_units;
      pos += n;
      row += n;
    }
    base += (kl + kPage - 1) / kPage;
  }
}

}  // namespace msa

using namespace msa;

extern "C" {

msa_status msa_kv_append(msa_plan_t plan, msa_rope_t rope, const int32_t* positions, const void* k,
                         int64_t k_row_stride, const void* v, int64_t v_row_stride, const int32_t* kv_indices,
                         void* k_pages, void* v_pages, float* k_scale, float* v_scale, msa_stream_t stream) {
  const char* fn = "msa_kv_append";
  if (!plan || !k || !v || !kv_indices || !k_pages || !v_pages)
    return set_error(MSA_ERR_INVALID_ARG, "%s: NULL argument", fn);
  const bool fp8 = plan->kv_dtype != MSA_KV_BF16;
  if (fp8 != (k_scale != nullptr) || fp8 != (v_scale != nullptr))
    return set_error(MSA_ERR_INVALID_ARG, "%s: k_scale/v_scale must be given exactly for FP8 K/V", fn);
  const int64_t width = int64_t(plan->hkv) * plan->d;
  msa_status s = check_append(fn, plan, rope, plan->d);
  if (s == MSA_OK) s = check_rows(fn, "k", k, k_row_stride, width);
  if (s == MSA_OK) s = check_rows(fn, "v", v, v_row_stride, width);
  if (s != MSA_OK) return s;
  if (!aligned16(k_pages) || !aligned16(v_pages))
    return set_error(MSA_ERR_INVALID_ARG, "%s: k_pages and v_pages must be 16-byte aligned", fn);
  if (k_pages == v_pages || (fp8 && k_scale == v_scale && plan->kv_dtype == MSA_KV_FP8_E4M3_BLOCK))
    return set_error(MSA_ERR_INVALID_ARG, "%s: K and V need pools and scales of their own", fn);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const KvAppendArgs a{reinterpret_cast<const AppendUnit*>(plan->aux_d + plan->append_units_off),
                       {static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v)},
                       {k_row_stride, v_row_stride},
                       {k_pages, v_pages},
                       {k_scale, v_scale},
                       positions,
                       kv_indices,
                       plan->num_pages,
                       plan->hkv,
                       {1, 1},
                       {1, 1},
                       0,
                       plan->err_d};
  const bool d128 = plan->d == 128;
  const auto launch =
      plan->kv_dtype == MSA_KV_BF16       ? (d128 ? launch_kv<128, MSA_KV_BF16> : launch_kv<64, MSA_KV_BF16>)
      : plan->kv_dtype == MSA_KV_FP8_E4M3 ? (d128 ? launch_kv<128, MSA_KV_FP8_E4M3> : launch_kv<64, MSA_KV_FP8_E4M3>)
                                          : (d128 ? launch_kv<128, MSA_KV_FP8_E4M3_BLOCK>
                                                  : launch_kv<64, MSA_KV_FP8_E4M3_BLOCK>);
  const cudaError_t e = launch(plan, table_of(rope), a, st);
  s = cuda_check(e, "msa_kv_append: launch");
  if (s == MSA_OK) s = scan_strided(plan, k, plan->total_q, width, k_row_stride, st);
  if (s == MSA_OK) s = scan_strided(plan, v, plan->total_q, width, v_row_stride, st);
  return s;
}

msa_status msa_pk_append(msa_plan_t plan, msa_rope_t rope, const int32_t* positions, const void* pk,
                         int64_t pk_row_stride, const int32_t* kv_indices, void* pk_pages, void* pk_pages_e4m3,
                         const float* pk_scale, void* pk_codes, void* pk_block_scales, const float* pk_global_scale,
                         msa_stream_t stream) {
  const char* fn = "msa_pk_append";
  if (!plan || !pk || !kv_indices) return set_error(MSA_ERR_INVALID_ARG, "%s: NULL argument", fn);
  if (!pk_pages && !pk_pages_e4m3 && !pk_codes)
    return set_error(MSA_ERR_INVALID_ARG, "%s: no pool to write", fn);
  if ((pk_pages_e4m3 != nullptr) != (pk_scale != nullptr))
    return set_error(MSA_ERR_INVALID_ARG, "%s: pk_scale goes with pk_pages_e4m3", fn);
  if ((pk_codes != nullptr) != (pk_block_scales != nullptr) || (pk_codes != nullptr) != (pk_global_scale != nullptr))
    return set_error(MSA_ERR_INVALID_ARG, "%s: pk_codes, pk_block_scales and pk_global_scale go together", fn);
  msa_status s = check_append(fn, plan, rope, plan->dp);
  if (s == MSA_OK) s = check_rows(fn, "pk", pk, pk_row_stride, plan->dp);
  if (s != MSA_OK) return s;
  if (!aligned16(pk_pages) || !aligned16(pk_pages_e4m3) || !aligned16(pk_codes) || !aligned16(pk_block_scales))
    return set_error(MSA_ERR_INVALID_ARG, "%s: the pools must be 16-byte aligned", fn);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const ProxyPools pools{static_cast<__nv_bfloat16*>(pk_pages), static_cast<uint8_t*>(pk_pages_e4m3), pk_scale,
                         static_cast<uint8_t*>(pk_codes), static_cast<uint8_t*>(pk_block_scales), pk_global_scale};
  auto run = [&](auto kernel) {
    const int rows = kPkThreads / (plan->dp / 16);
    return launch_pdl(kernel, dim3(plan->n_append_units, plan->decode ? 1 : 128 / rows), dim3(kPkThreads), 0, st,
                      table_of(rope),
                      reinterpret_cast<const AppendUnit*>(plan->aux_d + plan->append_units_off),
                      static_cast<const __nv_bfloat16*>(pk), pk_row_stride, positions, kv_indices, plan->num_pages,
                      pools, plan->err_d);
  };
  s = cuda_check(plan->dp == 64 ? run(pk_append_kernel<64>) : run(pk_append_kernel<32>), "msa_pk_append: launch");
  if (s == MSA_OK) s = scan_strided(plan, pk, plan->total_q, plan->dp, pk_row_stride, st);
  return s;
}

msa_status msa_append_bwd(msa_plan_t plan, msa_rope_t k_rope, msa_rope_t pk_rope, const int32_t* positions,
                          const int32_t* kv_indices, const float* dk_pages, const float* dv_pages,
                          const float* dpk_pages, float* dk, float* dv, float* dpk, msa_stream_t stream) {
  const char* fn = "msa_append_bwd";
  if (!plan || !kv_indices) return set_error(MSA_ERR_INVALID_ARG, "%s: NULL argument", fn);
  if ((dk_pages != nullptr) != (dk != nullptr) || (dv_pages != nullptr) != (dv != nullptr) ||
      (dpk_pages != nullptr) != (dpk != nullptr))
    return set_error(MSA_ERR_INVALID_ARG, "%s: gradient pages and rows go together", fn);
  if (!dk && !dv && !dpk) return set_error(MSA_ERR_INVALID_ARG, "%s: no gradient given", fn);
  if (plan->kv_dtype != MSA_KV_BF16) return set_error(MSA_ERR_UNSUPPORTED, "%s: bf16 K/V only", fn);
  msa_status s = check_append(fn, plan, k_rope, plan->d);
  if (s == MSA_OK) s = check_append(fn, plan, pk_rope, plan->dp);
  if (s != MSA_OK) return s;
  if (!aligned16(dk_pages) || !aligned16(dv_pages) || !aligned16(dpk_pages) || !aligned16(dk) || !aligned16(dv) ||
      !aligned16(dpk))
    return set_error(MSA_ERR_INVALID_ARG, "%s: gradients must be 16-byte aligned", fn);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const GradSet gk{dk_pages, dk, dk ? plan->hkv : 0, plan->d}, gv{dv_pages, dv, dv ? plan->hkv : 0, plan->d},
      gp{dpk_pages, dpk, dpk ? 1 : 0, plan->dp};
  s = cuda_check(launch_pdl(append_bwd_kernel, dim3(plan->n_append_units, gk.heads + gv.heads + gp.heads),
                            dim3(kThreads), 0, st, table_of(k_rope), table_of(pk_rope),
                            reinterpret_cast<const AppendUnit*>(plan->aux_d + plan->append_units_off), positions,
                            kv_indices, plan->num_pages, gk, gv, gp, plan->err_d),
                 "msa_append_bwd: launch");
  const int64_t rows = plan->total_q;
  if (s == MSA_OK) s = scan_rows(plan, dk, rows * plan->hkv * plan->d, 4, st);
  if (s == MSA_OK) s = scan_rows(plan, dv, rows * plan->hkv * plan->d, 4, st);
  if (s == MSA_OK) s = scan_rows(plan, dpk, rows * plan->dp, 4, st);
  return s;
}

}  // extern "C"
