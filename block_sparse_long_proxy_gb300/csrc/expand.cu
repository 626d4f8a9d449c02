// The expanded form of a latent cache: K and V pages for msa_sparse_attn out of
// pages of [latent | rotated part] rows,
//   K[h] = [w_k[h] . latent | rotated part],  V[h] = w_v[h] . latent.
//
// A matrix product of the page's 128 rows with the head's rows of w_k and w_v
// together (N = nope + d <= 240), on tcgen05, fp32 in tensor memory, rounded once
// to bf16.  A unit is (page-table entry, a few heads): the page's latents stay in
// shared memory (128 KB at 512) while the heads' weights stream past, 64 dims a
// stage.  Persistent: warps 0-3 write K and 4-7 V out of one of two
// accumulators, a thread being a key, while the next head's products fill the
// other.
#include <algorithm>

#include "msa_internal.h"
#include "ptx.cuh"

namespace msa {
namespace {

constexpr int kThreads = 352;        // 8 epilogue warps, B producer, MMA, A producer
constexpr int kABytes = 8 * 16384;
constexpr int kMaxStages = 8;
constexpr int kRing = 92160;         // weights: 3 stages at the widest (240 rows)
constexpr int kBarOff = kABytes + kRing;
constexpr int kSmem = kBarOff + 512;

struct ExpandArgs {
  const __nv_bfloat16* latent;
  const int32_t* kv_indices;
  const int32_t* keys;    // keys of each entry's page, 1..128
  __nv_bfloat16* k_pages;
  __nv_bfloat16* v_pages;
  uint32_t* err;
  int64_t num_pages;
  int32_t entries, heads, per_unit, groups;
  int32_t chunks;         // latent_dim / 64
  int32_t width;          // of a cache row
  int32_t nope, d, rope;
  int32_t stages;
};

__global__ void __launch_bounds__(kThreads, 1)
    expand_kernel(const __grid_constant__ CUtensorMap c_map, const __grid_constant__ CUtensorMap wk_map,
                  const __grid_constant__ CUtensorMap wv_map, const ExpandArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* a_full = bars;               // [8]: a chunk of the unit's latents
  uint64_t* a_empty = a_full + 8;        // [8]
  uint64_t* b_full = a_empty + 8;        // [stages]
  uint64_t* b_empty = b_full + kMaxStages;
  uint64_t* d_full = b_empty + kMaxStages;  // [2] accumulators
  uint64_t* d_empty = d_full + 2;           // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(d_empty + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = a.nope + a.d, stage_bytes = n * 128;
  if (threadIdx.x == 0) {
    prefetch_tmap(&c_map);
    prefetch_tmap(&wk_map);
    prefetch_tmap(&wv_map);
    for (int i = 0; i < 8; ++i) mbar_init(a_full + i, 1), mbar_init(a_empty + i, 1);
    for (int i = 0; i < kMaxStages; ++i) mbar_init(b_full + i, 1), mbar_init(b_empty + i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(d_full + i, 1), mbar_init(d_empty + i, 8);
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const int units = a.entries * a.groups;
  auto head0 = [&](int u) { return u % a.groups * a.per_unit; };
  auto heads_of = [&](int u) { return min(a.per_unit, a.heads - head0(u)); };
  // a page outside the pool: its unit computes on page 0 and writes nothing
  auto page_of = [&](int u, bool& good) {
    const int64_t page = a.kv_indices[u / a.groups];
    good = page >= 0 && page < a.num_pages;
    return good ? page : int64_t(0);
  };

  if (warp == 10) {
    if (lane == 0) {
      bool ok = true, good;
      for (int k = 0, u = blockIdx.x; u < units && ok; ++k, u += gridDim.x) {
        const int row = static_cast<int>(page_of(u, good) * 128);
        for (int c = 0; c < a.chunks && ok; ++c) {
          if (!(ok = mbar_wait(a_empty + c, (k & 1) ^ 1, a.err))) break;
          mbar_expect_tx(a_full + c, 16384);
          tma_load_2d(smem + c * 16384, &c_map, a_full + c, c * 64, row);
        }
      }
    }
  } else if (warp == 8) {
    if (lane == 0) {
      bool ok = true;
      int it = 0;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x)
        for (int h = head0(u), h1 = h + heads_of(u); h < h1 && ok; ++h)
          for (int c = 0; c < a.chunks && ok; ++c, ++it) {
            const int s = it % a.stages;
            if (!(ok = mbar_wait(b_empty + s, (it / a.stages & 1) ^ 1, a.err))) break;
            uint8_t* dst = smem + kABytes + s * stage_bytes;
            mbar_expect_tx(b_full + s, stage_bytes);
            tma_load_2d(dst, &wk_map, b_full + s, c * 64, h * a.nope);
            tma_load_2d(dst + a.nope * 128, &wv_map, b_full + s, c * 64, h * a.d);
          }
    }
  } else if (warp == 9) {
    if (lane == 0) {
      const uint32_t id = idesc_bf16_f32(128, n, false, false);
      const uint64_t ad = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128);
      bool ok = true;
      int it = 0, acc = 0;
      for (int k = 0, u = blockIdx.x; u < units && ok; ++k, u += gridDim.x) {
        const int heads = heads_of(u);
        for (int h = 0; h < heads && ok; ++h, ++acc) {
          const uint32_t d = tmem + (acc & 1) * 256;
          if (!(ok = mbar_wait(d_empty + (acc & 1), (acc >> 1 & 1) ^ 1, a.err))) break;
          for (int c = 0; c < a.chunks; ++c, ++it) {
            const int s = it % a.stages;
            if (h == 0 && !(ok = mbar_wait(a_full + c, k & 1, a.err))) break;
            if (!(ok = mbar_wait(b_full + s, it / a.stages & 1, a.err))) break;
            tc_fence_after();
            const uint64_t bd = smem_desc(smem_u32(smem + kABytes + s * stage_bytes), 16, 1024, kSwizzle128);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ss(d, ad + ((c * 16384 + kk * 32) >> 4), bd + ((kk * 32) >> 4), id, c > 0 || kk > 0);
            mma_commit(b_empty + s);
            if (h == heads - 1) mma_commit(a_empty + c);
          }
          if (ok) mma_commit(d_full + (acc & 1));
        }
      }
    }
  } else {
    const int which = warp >> 2, r = (warp & 3) * 32 + lane;  // 0: K, 1: V
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    int acc = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      bool good;
      const int64_t page = page_of(u, good);
      if (!good && threadIdx.x == 0) atomicOr(a.err, kErrDeviceCheck);
      const bool mine = good && r < a.keys[u / a.groups];
      uint4 tail[8];  // the rotated part, the same for every head
      if (which == 0 && mine) {
        const uint4* src = reinterpret_cast<const uint4*>(a.latent + (page * 128 + r) * a.width + a.chunks * 64);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < a.rope / 8) tail[c] = src[c];
      }
      const int cols = which == 0 ? a.nope : a.d;
      for (int h = head0(u), h1 = h + heads_of(u); h < h1; ++h, ++acc) {
        if (ok) ok = mbar_wait(d_full + (acc & 1), acc >> 1 & 1, a.err);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        const uint32_t at = tmem + (acc & 1) * 256 + lane_base + (which == 0 ? 0 : a.nope);
        float* dst = reinterpret_cast<float*>((which == 0 ? a.k_pages : a.v_pages) + ((page * a.heads + h) * 128 + r) * a.d);
        for (int c = 0; c < cols / 16; ++c) {
          uint32_t v[16];
          tmem_ld16(at + 16 * c, v);
          tmem_wait_ld();
          if (!mine || !ok) continue;
          float w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = __uint_as_float(pack_bf16x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])));
          st_global_v8(dst + 8 * c, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(d_empty + (acc & 1));
        if (which == 0 && mine && ok) {
#pragma unroll
          for (int c = 0; c < 8; c += 2)
            if (c < a.rope / 8) {
              const uint32_t* x = &tail[c].x;
              const uint32_t* y = &tail[c + 1].x;
              st_global_v8(dst + a.nope / 2 + 4 * c, __uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]),
                           __uint_as_float(x[3]), __uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]),
                           __uint_as_float(y[3]));
            }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Heads a unit: the fewest rounds of the persistent grid, a unit's start
// counting as a head and a half.
int heads_per_unit(int64_t entries, int heads, int sms) {
  int best = heads;
  double least = 1e300;
  for (int groups = 1; groups <= heads; ++groups) {
    const int per = (heads + groups - 1) / groups;
    const int64_t units = entries * ((heads + per - 1) / per);
    const double t = static_cast<double>((units + sms - 1) / sms) * (per + 1.5);
    if (t < least) least = t, best = per;
  }
  return best;
}

msa_status launch_expand(const msa_plan_s* p, const void* latent_pages, const void* w_k, const void* w_v,
                         const int32_t* kv_indices, int32_t latent_dim, int32_t rope_dim, void* k_pages, void* v_pages,
                         cudaStream_t st) {
  const int width = latent_dim + rope_dim, nope = p->d - rope_dim;
  CUtensorMap cm, km, vm;
  auto rows = [](CUtensorMap* m, const void* base, int64_t n, int wide, int box_rows) {
    const uint64_t dims[2] = {static_cast<uint64_t>(wide), static_cast<uint64_t>(n)};
    const uint64_t str[1] = {static_cast<uint64_t>(wide) * 2};
    const uint32_t box[2] = {64, static_cast<uint32_t>(box_rows)};
    return encode_tensor_map(m, 2, base, dims, str, box, 1, 128);
  };
  if (!rows(&cm, latent_pages, p->num_pages * 128, width, 128) || !rows(&km, w_k, int64_t(p->hkv) * nope, latent_dim, nope) ||
      !rows(&vm, w_v, int64_t(p->hkv) * p->d, latent_dim, p->d))
    return set_error(MSA_ERR_CUDA, "msa_latent_expand: tensor map encoding failed");
  ExpandArgs a{};
  a.latent = static_cast<const __nv_bfloat16*>(latent_pages);
  a.kv_indices = kv_indices;
  a.keys = p->aux_d + p->entry_keys_off;
  a.k_pages = static_cast<__nv_bfloat16*>(k_pages);
  a.v_pages = static_cast<__nv_bfloat16*>(v_pages);
  a.err = p->err_d;
  a.num_pages = p->num_pages;
  a.entries = p->n_page_entries;
  a.heads = p->hkv;
  a.per_unit = heads_per_unit(a.entries, p->hkv, p->num_sms);
  a.groups = (p->hkv + a.per_unit - 1) / a.per_unit;
  a.chunks = latent_dim / 64;
  a.width = width;
  a.nope = nope, a.d = p->d, a.rope = rope_dim;
  a.stages = std::min(kMaxStages, kRing / ((nope + p->d) * 128));
  const int64_t units = int64_t(a.entries) * a.groups;
  if (units > 0x7FFFFFFF) return set_error(MSA_ERR_UNSUPPORTED, "msa_latent_expand: too many pages");
  const int smem = kSmem + 1024;
  cudaError_t e = cudaFuncSetAttribute(expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = launch_pdl(expand_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(units, p->num_sms))), dim3(kThreads), smem, st,
                   cm, km, vm, a);
  return cuda_check(e, "msa_latent_expand: launch");
}

}  // namespace

// Keys of each page-table entry's page: 128, and what is left in a sequence's last (bf16 plans).
void expand_plan_tables(msa_plan_s* p, std::vector<int32_t>& aux) {
  if (p->kv_dtype != MSA_KV_BF16) return;
  p->entry_keys_off = static_cast<int64_t>(aux.size());
  for (int32_t k : p->kv_lens)
    for (int32_t left = k; left > 0; left -= std::min(left, kPage)) aux.push_back(std::min(left, kPage));
}

}  // namespace msa

using namespace msa;

extern "C" msa_status msa_latent_expand(msa_plan_t plan, const void* latent_pages, const void* w_k, const void* w_v,
                                        const int32_t* kv_indices, int32_t latent_dim, int32_t rope_dim, void* k_pages,
                                        void* v_pages, msa_stream_t stream) {
  const char* fn = "msa_latent_expand";
  if (!plan || !latent_pages || !w_k || !w_v || !kv_indices || !k_pages || !v_pages)
    return set_error(MSA_ERR_INVALID_ARG, "%s: NULL argument", fn);
  msa_status s = check_latent_dims(fn, latent_dim, rope_dim);
  if (s != MSA_OK) return s;
  if (plan->kv_dtype != MSA_KV_BF16) return set_error(MSA_ERR_UNSUPPORTED, "%s: bf16 K/V only", fn);
  if (rope_dim >= plan->d)
    return set_error(MSA_ERR_INVALID_ARG, "%s: rope_dim %d leaves nothing of head_dim %d", fn, rope_dim, plan->d);
  auto aligned = [](const void* x, unsigned n) { return (reinterpret_cast<uintptr_t>(x) & (n - 1)) == 0; };
  if (!aligned(latent_pages, 16) || !aligned(w_k, 16) || !aligned(w_v, 16) || !aligned(k_pages, 32) || !aligned(v_pages, 32))
    return set_error(MSA_ERR_INVALID_ARG, "%s: inputs must be 16-byte aligned and the K/V pages 32-byte aligned", fn);
  if (k_pages == v_pages) return set_error(MSA_ERR_INVALID_ARG, "%s: K and V need pools of their own", fn);
  if ((s = check_device(fn, plan)) != MSA_OK) return s;
  return launch_expand(plan, latent_pages, w_k, w_v, kv_indices, latent_dim, rope_dim, k_pages, v_pages,
                       reinterpret_cast<cudaStream_t>(stream));
}
