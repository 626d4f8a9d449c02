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

// four e4m3 codes times a factor, rounded to e4m3 again
__device__ __forceinline__ uint32_t rescale4(uint32_t v, float f) {
  const uint32_t a = e4m3x2_to_f16x2(v), b = e4m3x2_to_f16x2(v >> 16);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return e4m3x4(x.x * f, x.y * f, y.x * f, y.y * f);
}

// K (blockIdx.z 0, rotated) or V (1) of one page and one KV head.
template <int D, msa_kv_dtype KIND>
__global__ void __launch_bounds__(kThreads)
    kv_append_kernel(const __grid_constant__ RopeTable tab, const AppendUnit* __restrict__ units,
                     const __nv_bfloat16* __restrict__ k, int64_t k_stride, const __nv_bfloat16* __restrict__ v,
                     int64_t v_stride, const int32_t* __restrict__ positions, const int32_t* __restrict__ kv_indices,
                     int64_t num_pages, void* __restrict__ k_pages, void* __restrict__ v_pages, float* k_scale,
                     float* v_scale, int32_t hkv, uint32_t* err) {
  pdl_wait();
  constexpr int kChunks = D / 16, kRows = kThreads / kChunks, kPasses = 128 / kRows;
  const AppendUnit u = units[blockIdx.x];
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z == 1;
  const int64_t page = kv_indices[u.entry];
  if (page < 0 || page >= num_pages) {
    if (threadIdx.x == 0) atomicOr(err, kErrDeviceCheck);
    return;
  }
  const int slot0 = u.slot0_n & 0xFF, n = u.slot0_n >> 8;
  const int c = threadIdx.x % kChunks, r0 = threadIdx.x / kChunks;
  RopeChunk ch = rope_chunk(tab, c);
  if (is_v || !ch.rotated) ch = {16 * c, 16 * c + 8, false};
  const __nv_bfloat16* src = (is_v ? v + u.row * v_stride : k + u.row * k_stride) + h * D;
  const int64_t stride = is_v ? v_stride : k_stride;
  const int64_t head_row = (page * hkv + h) * 128;  // first row of the (page, head) in the pool

  float x[kPasses][16];
  float amax = 0.f;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int i = p * kRows + r0;
    if (i < n) {
      load8(src + i * stride + ch.lo, x[p]);
      load8(src + i * stride + ch.hi, x[p] + 8);
      if (ch.rotated) {
        float cs[8], sn[8];
        rope_angles(tab, c, positions ? positions[u.row + i] : u.pos + i, false, cs, sn);
        rope_rotate(tab.interleaved != 0, cs, sn, x[p]);
      }
      if (KIND == MSA_KV_FP8_E4M3_BLOCK) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float a = fabsf(x[p][e]);
          if (a <= 3.4028234e38f) amax = fmaxf(amax, a);  // infinities saturate, they set no scale
        }
      }
    }
  }
  if (KIND == MSA_KV_BF16) {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? v_pages : k_pages) + (head_row + slot0) * D;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int i = p * kRows + r0;
      if (i < n) {
        store8(dst + i * D + ch.lo, x[p]);
        store8(dst + i * D + ch.hi, x[p] + 8);
      }
    }
    return;
  }
  uint8_t* pool = static_cast<uint8_t*>(is_v ? v_pages : k_pages) + head_row * D;
  float* scales = is_v ? v_scale : k_scale;
  float by = 1.f;  // the codes are x * by (block) or x / by (one scale a head)
  if (KIND == MSA_KV_FP8_E4M3_BLOCK) {
    __shared__ float warp_max[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, warp_max[w]);
    int e = block_exp(amax);
    float* sp = scales + page * hkv + h;
    if (slot0 > 0) {  // rows came before: the scale only grows
      const float old = *sp;
      if (!(old > 0.f && old <= pow2(kMaxExp))) {  // never written: the old slots keep their bytes
        if (threadIdx.x == 0) atomicOr(err, kErrDeviceCheck);
      } else {
        // another writer's scale need not be a power of two: round it up to one
        const uint32_t ou = __float_as_uint(old);
        e = max(e, static_cast<int>(ou >> 23) - 127 + ((ou & 0x7FFFFFu) != 0u ? 1 : 0));
        const float f = old * pow2(-e);
        if (f != 1.f) {
          uint4* q = reinterpret_cast<uint4*>(pool);
          for (int i = threadIdx.x; i < slot0 * (D / 16); i += kThreads) {
            uint4 w = q[i];
            w.x = rescale4(w.x, f), w.y = rescale4(w.y, f), w.z = rescale4(w.z, f), w.w = rescale4(w.w, f);
            q[i] = w;
          }
        }
      }
      __syncthreads();  // every thread has read the old scale
    }
    if (threadIdx.x == 0) *sp = pow2(e);
    by = pow2(-e);
  } else {
    by = scales[h];
  }
  uint8_t* dst = pool + slot0 * D;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int i = p * kRows + r0;
    if (i < n) {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[p][e] = KIND == MSA_KV_FP8_E4M3_BLOCK ? x[p][e] * by : __fdiv_rn(x[p][e], by);
      *reinterpret_cast<uint2*>(dst + i * D + ch.lo) = e4m3x8(x[p]);
      *reinterpret_cast<uint2*>(dst + i * D + ch.hi) = e4m3x8(x[p] + 8);
    }
  }
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

template <int DP>
__global__ void __launch_bounds__(kThreads)
    pk_append_kernel(const __grid_constant__ RopeTable tab, const AppendUnit* __restrict__ units,
                     const __nv_bfloat16* __restrict__ pk, int64_t stride, const int32_t* __restrict__ positions,
                     const int32_t* __restrict__ kv_indices, int64_t num_pages,
                     const __grid_constant__ ProxyPools pools, uint32_t* err) {
  pdl_wait();
  constexpr int kChunks = DP / 16, kRows = kThreads / kChunks;
  __shared__ __align__(16) float rows[kRows][DP];  // rotated: NVFP4 blocks are 16 consecutive dims
  const AppendUnit u = units[blockIdx.x];
  const int64_t page = kv_indices[u.entry];
  if (page < 0 || page >= num_pages) {
    if (threadIdx.x == 0) atomicOr(err, kErrDeviceCheck);
    return;
  }
  const int slot0 = u.slot0_n & 0xFF, n = u.slot0_n >> 8;
  const int c = threadIdx.x % kChunks, r = threadIdx.x / kChunks;
  const RopeChunk ch = rope_chunk(tab, c);
  const float fp8_scale = pools.e4m3 ? *pools.e4m3_scale : 1.f;
  const float g = pools.codes ? *pools.global_scale : 1.f;
  for (int base = 0; base < n; base += kRows) {
    const int i = base + r;
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
      const int64_t at = (page * 128 + slot0 + i) * DP;
      if (pools.bf16) {
        store8(pools.bf16 + at + ch.lo, x);
        store8(pools.bf16 + at + ch.hi, x + 8);
      }
      if (pools.codes) {
        store8(&rows[r][ch.lo], x);
        store8(&rows[r][ch.hi], x + 8);
      }
      if (pools.e4m3) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __fdiv_rn(x[e], fp8_scale);
        *reinterpret_cast<uint2*>(pools.e4m3 + at + ch.lo) = e4m3x8(x);
        *reinterpret_cast<uint2*>(pools.e4m3 + at + ch.hi) = e4m3x8(x + 8);
      }
    }
    if (pools.codes) {
      __syncthreads();
      if (i < n) {
        load8(&rows[r][16 * c], x);
        load8(&rows[r][16 * c + 8], x + 8);
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
        const uint32_t sc = nvfp4_block_scale(amax, g);
        const float bs = e4m3_value(sc);
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e >> 3] |= (bs > 0.f ? nvfp4_code(x[e], bs, g) : 0u) << (4 * (e & 7));
        const int64_t row = page * 128 + slot0 + i;
        *reinterpret_cast<uint2*>(pools.codes + row * (DP / 2) + 8 * c) = make_uint2(w[0], w[1]);
        pools.block_scales[row * kChunks + c] = static_cast<uint8_t>(sc);
      }
      __syncthreads();
    }
  }
}

// Gradient pages to rows: dK (rotated back), dV and dpk (rotated back).
// blockIdx.y: KV heads of K, then of V, then the proxy head.
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
      rope_angles(tab, c, positions ? positions[u.row + i] : u.pos + i, true, cs, sn);
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
  int dev = 0;
  const msa_status s = cuda_check(cudaGetDevice(&dev), fn);
  if (s != MSA_OK) return s;
  if (dev != plan->device)
    return set_error(MSA_ERR_INVALID_ARG, "%s: the plan belongs to device %d, device %d is current", fn,
                     plan->device, dev);
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

template <int D, msa_kv_dtype KIND, typename... A>
cudaError_t launch_kv(const msa_plan_s* p, cudaStream_t st, A... a) {
  return launch_pdl(kv_append_kernel<D, KIND>, dim3(p->n_append_units, p->hkv, 2), dim3(kThreads), 0, st, a...);
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
  auto run = [&](auto launch) {
    return launch(plan, st, table_of(rope), reinterpret_cast<const AppendUnit*>(plan->aux_d + plan->append_units_off),
                  static_cast<const __nv_bfloat16*>(k), k_row_stride, static_cast<const __nv_bfloat16*>(v),
                  v_row_stride, positions, kv_indices, plan->num_pages, k_pages, v_pages, k_scale, v_scale, plan->hkv,
                  plan->err_d);
  };
  const bool d128 = plan->d == 128;
  cudaError_t e;
  if (plan->kv_dtype == MSA_KV_BF16)
    e = run([&](auto... a) { return d128 ? launch_kv<128, MSA_KV_BF16>(a...) : launch_kv<64, MSA_KV_BF16>(a...); });
  else if (plan->kv_dtype == MSA_KV_FP8_E4M3)
    e = run([&](auto... a) {
      return d128 ? launch_kv<128, MSA_KV_FP8_E4M3>(a...) : launch_kv<64, MSA_KV_FP8_E4M3>(a...);
    });
  else
    e = run([&](auto... a) {
      return d128 ? launch_kv<128, MSA_KV_FP8_E4M3_BLOCK>(a...) : launch_kv<64, MSA_KV_FP8_E4M3_BLOCK>(a...);
    });
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
    return launch_pdl(kernel, dim3(plan->n_append_units), dim3(kThreads), 0, st, table_of(rope),
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
