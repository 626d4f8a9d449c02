// The expanded form of a latent cache: K and V pages for msa_sparse_attn out of
// pages of [latent | rotated part] rows,
//   K[h] = [w_k[h] . latent | rotated part],  V[h] = w_v[h] . latent.
//
// A matrix product of two pages' 256 rows with the head's rows of w_k and w_v
// together (nope + d <= 240, N the next multiple of 32), on tcgen05 by pairs of SMs
// (cta_group::2), fp32 in tensor memory, rounded once to bf16.  A unit is (two page-table entries, a few
// heads): each CTA of a pair keeps its page's latents in shared memory (128 KB
// at 512) while the heads' weights stream past, 64 dims a stage, of which each CTA
// loads one half of the N rows for both: an SM reads 98 KB of weights a head
// where one by itself reads 196.
// Persistent: warps 0-3 write K and 4-7 V out of one of two
// accumulators, a thread being a key, while the next head's products fill the
// other.
//
// 32768 rows, 32 heads, 64 + 64 dims, latent 512 (581 MB, 206 GFLOP of products):
// 137 us (133 to 143 by the GPU), 4.2 TB/s and 1.5 PFLOP/s (154 in passes without a
// pause, at the power limit).  The products are 0.8 of it; the rest is the
// issuing thread's waits between them and the stores, which at latent 128 take
// 116 us alone.  One CTA a page: 241 us.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "msa_internal.h"
#include "ptx.cuh"

namespace msa {
namespace {

constexpr int kThreads = 352;        // 8 epilogue warps, B producer, MMA, A producer
constexpr int kABytes = 8 * 16384;
constexpr int kMaxStages = 8;
constexpr int kRing = 98304;         // half the weights, 128 dims a stage: 3 stages at the widest (128 rows)
constexpr int kBarOff = kABytes + kRing;
constexpr int kSmem = kBarOff + 512;

// ---- pairs of CTAs
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Arrive on CTA 0's barrier at the same place as `bar`: what is handed over is tensor
// memory that was read.  The next product may overwrite it by the rules of tensor
// memory, which need no release: tcgen05.wait::ld has ended the reads,
// tcgen05.fence::before_thread_sync orders them before the arrive, and
// tcgen05.fence::after_thread_sync the issuing thread's products behind its wait; a
// relaxed arrive and the wait that sees it are the order between the two threads.  (A
// release would also wait for the warp's stores to K and V: 152 us where this took 139.)
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
// mbar_wait_inl for a barrier on which the other CTA arrives (the clock is read
// after a poll that failed only: it takes about a microsecond)
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, uint32_t* err) {
  uint64_t t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(100000u)
        : "memory");
    if (ok) return true;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitLimitNs) {
      atomicOr(err, kErrTimeout);
      return false;
    }
  }
}
// D (256 rows, 128 a CTA) (+)= A (128 rows a CTA) * B^T (half of N rows a CTA), by the lane that has `leader`
__device__ __forceinline__ void mma_pair(bool leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(leader))
      : "memory");
}
// A load into this CTA's shared memory that counts on CTA 0's barrier, at the same
// place as `bar`: its thread, which issues for both, waits for the bytes of both.
// (A thread of CTA 1 that passed on what its own barrier said took 1100 clocks a
// stage, most of them for the release of a remote arrive.)
__device__ __forceinline__ void tma_load_pair(void* dst, const void* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, 0;\n\t"
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [a];\n\t}" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}
// arrives on both CTAs' barriers (or those in `ctas`) when the products issued so far are complete
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t ctas = 3) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(ctas)
      : "memory");
}

// N of a head's products: its rows of w_k and w_v together, to the next multiple of
// 32, which pairs of SMs with 256 rows take.  CTA 0 has the first half of N, CTA 1 the
// other rows; what is behind them in its shared memory goes to columns that nobody reads.
constexpr int product_cols(int nope, int d) { return (nope + d + 31) / 32 * 32; }

struct ExpandArgs {
  const __nv_bfloat16* latent;
  const int32_t* kv_indices;
  const uint8_t* keys;    // keys of each entry's page, 1..128
  __nv_bfloat16* k_pages;
  __nv_bfloat16* v_pages;
  uint32_t* err;
  int64_t num_pages;
  int32_t entries, pairs, heads, per_unit, groups;
  int32_t chunks;         // latent_dim / 64, two a step
  int32_t width;          // of a cache row
  int32_t stages;
};

template <int D, int ROPE>
__global__ void __launch_bounds__(kThreads, 1)
    expand_kernel(const __grid_constant__ CUtensorMap c_map, const __grid_constant__ CUtensorMap wk_map,
                  const __grid_constant__ CUtensorMap wv0_map, const __grid_constant__ CUtensorMap wv1_map,
                  const ExpandArgs a) {
  constexpr int kNope = D - ROPE, n = product_cols(kNope, D), half = n / 2, chunk_bytes = half * 128, stage_bytes = 2 * chunk_bytes;
  static_assert(n % 32 == 0 && n <= 256, "N of a product by a pair of SMs; 256 columns an accumulator");
  static_assert(half > kNope && half % 8 == 0 && kNope % 8 == 0 && half <= kNope + D, "boxes of whole swizzled groups of rows");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the same place in both CTAs of the pair: their windows start alike
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* a_full = bars;               // [8] CTA 0: a chunk of both pages' latents
  uint64_t* a_empty = a_full + 8;        // [8]
  uint64_t* b_full = a_empty + 8;        // [stages] CTA 0: both halves
  uint64_t* b_empty = b_full + kMaxStages;
  uint64_t* d_full = b_empty + kMaxStages;  // [2] accumulators
  uint64_t* d_empty = d_full + 2;           // [2] CTA 0: read, by the warps of both
  uint64_t* drain = d_empty + 2;            // CTA 0: every product issued is complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = cta_rank();
  if (threadIdx.x == 0) {
    prefetch_tmap(&c_map);
    prefetch_tmap(&wk_map);
    prefetch_tmap(&wv0_map);
    prefetch_tmap(&wv1_map);
    for (int i = 0; i < 8; ++i) mbar_init(a_full + i, 1), mbar_init(a_empty + i, 1);
    for (int i = 0; i < kMaxStages; ++i) mbar_init(b_full + i, 1), mbar_init(b_empty + i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(d_full + i, 1), mbar_init(d_empty + i, 16);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const int steps = a.chunks / 2;
  const int units = a.pairs * a.groups, unit0 = blockIdx.x / 2, step = gridDim.x / 2;
  auto head0 = [&](int u) { return u % a.groups * a.per_unit; };
  auto heads_of = [&](int u) { return min(a.per_unit, a.heads - head0(u)); };
  // The unit's heads in turn, another first for each pair of pages, and a head's
  // dims from a place of its own on, so that units side by side read different
  // weights.  The order of a sum goes by its head alone: a page named twice gets
  // the same bits.
  auto head_of = [&](int u, int i) { return head0(u) + (i + u / a.groups) % heads_of(u); };
  // (the loops below count stages and dims up: a division by a run-time number
  // takes about 100 clocks, and three of them for 64 dims were half of their 1000)
  struct Ring {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
      if (++s == n) s = 0, phase ^= 1;
    }
    __device__ __forceinline__ void back(int n) {
      if (--s < 0) s = n - 1, phase ^= 1;
    }
  };
  // this CTA's entry of the pair's two, and its page; none, or a page outside the
  // pool: it computes on page 0 and writes nothing
  auto entry_of = [&](int u) { return u / a.groups * 2 + rank; };
  auto page_of = [&](int u, bool& good) {
    const int e = entry_of(u);
    const int64_t page = e < a.entries ? a.kv_indices[e] : -1;
    good = page >= 0 && page < a.num_pages;
    return good ? page : int64_t(0);
  };

  if (warp == 10) {
    if (lane == 0) {
      bool ok = true, good;
      uint32_t have = 0, odd = 0;  // chunks that were loaded, and the phase of the last time
      for (int k = 0, u = unit0; u < units && ok; ++k, u += step) {
        const int row = static_cast<int>(page_of(u, good) * 128);
        for (int i = 0, c = head_of(u, 0) % steps; i < steps && ok; ++i, c = c + 1 == steps ? 0 : c + 1) {
          if (!(ok = wait_cluster(a_empty + c, (k & 1) ^ 1, a.err))) break;
          if (rank == 0) mbar_expect_tx(a_full + c, 4 * 16384);
          for (int e = 0; e < 2; ++e) tma_load_pair(smem + (2 * c + e) * 16384, &c_map, a_full + c, (2 * c + e) * 64, row);
          have |= 1u << c, odd = (odd & ~(1u << c)) | static_cast<uint32_t>(k & 1) << c;
        }
      }
      // Nothing is under way to either CTA's shared memory when they leave, although a role
      // that gave up a wait leaves loads unused.
      for (int c = 0; rank == 0 && c < steps; ++c)
        if (have >> c & 1u) mbar_wait_inl(a_full + c, odd >> c & 1u, a.err);
    }
  } else if (warp == 8) {
    if (lane == 0) {
      bool ok = true;
      Ring ring;
      int loads = 0;
      for (int u = unit0; u < units && ok; u += step)
        for (int i = 0; i < heads_of(u) && ok; ++i) {
          const int h = head_of(u, i);
          for (int j = 0, c = h % steps; j < steps && ok; ++j, c = c + 1 == steps ? 0 : c + 1, ring.next(a.stages)) {
            const int s = ring.s;
            if (!(ok = wait_cluster(b_empty + s, ring.phase ^ 1, a.err))) break;
            uint8_t* dst = smem + kABytes + s * stage_bytes;
            if (rank == 0) mbar_expect_tx(b_full + s, 2 * (kNope + D) * 128);
            for (int e = 0; e < 2; ++e, dst += chunk_bytes) {
              const int x = (2 * c + e) * 64;
              if (rank == 0) {  // w_k's rows and the first of w_v's
                tma_load_pair(dst, &wk_map, b_full + s, x, h * kNope);
                tma_load_pair(dst + kNope * 128, &wv0_map, b_full + s, x, h * D);
              } else {
                tma_load_pair(dst, &wv1_map, b_full + s, x, h * D + half - kNope);
              }
            }
            loads = min(loads + 1, a.stages);
          }
        }
      for (; rank == 0 && loads > 0; --loads) {  // (as the latents)
        ring.back(a.stages);
        mbar_wait_inl(b_full + ring.s, ring.phase, a.err);
      }
    }
  } else if (warp == 9) {
    if (rank == 0) {  // issues for both CTAs: the whole warp goes through the loop, one elected lane issuing
      const uint32_t id = idesc_bf16_f32(256, n, false, false);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint64_t ad = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128);
      const uint64_t bd0 = smem_desc(smem_u32(smem + kABytes), 16, 1024, kSwizzle128);
      const bool leader = elect_one();
      bool ok = true;
      auto all = [&](bool done) { return static_cast<bool>(__all_sync(0xFFFFFFFFu, done)); };
      Ring ring;
      int acc = 0;
      for (int k = 0, u = unit0; u < units && ok; ++k, u += step) {
        const int heads = heads_of(u);
        for (int i = 0; i < heads && ok; ++i, ++acc) {
          const int h = head_of(u, i);
          const uint32_t d = tm + (acc & 1) * 256;
          if (!(ok = all(wait_cluster(d_empty + (acc & 1), (acc >> 1 & 1) ^ 1, a.err)))) break;
          for (int j = 0, c = h % steps; j < steps; ++j, c = c + 1 == steps ? 0 : c + 1, ring.next(a.stages)) {
            const int s = ring.s;
            if (i == 0 && !(ok = all(mbar_wait_inl(a_full + c, k & 1, a.err)))) break;
            if (!(ok = all(mbar_wait_inl(b_full + s, ring.phase, a.err)))) break;
            tc_fence_after();
            const uint64_t bd = bd0 + s * (stage_bytes >> 4), ac = ad + c * (32768 >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_pair(leader, d, ac + ((kk / 4 * 16384 + kk % 4 * 32) >> 4), bd + ((kk / 4 * chunk_bytes + kk % 4 * 32) >> 4),
                       id, j > 0 || kk > 0);
            if (leader) {
              commit_pair(b_empty + s);
              if (i == heads - 1) commit_pair(a_empty + c);
            }
          }
          if (ok && leader) commit_pair(d_full + (acc & 1));
        }
      }
      if (leader) commit_pair(drain, 1);  // nor a product, also after a wait that was given up
      all(mbar_wait_inl(drain, 0, a.err));
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // Four lanes hold 64 consecutive bytes of a row, or two hold 32, when they
    // store: with a row a lane, in 32-byte sectors, the stores alone took 143 us
    // (and by TMA out of boxes of 64 columns 200 us, mostly waits for the boxes).
    const int which = warp >> 2, row0 = (warp & 3) * 32, quad = lane >> 2, j = lane & 3;  // 0: K, 1: V
    const uint32_t lane_base = static_cast<uint32_t>(row0) << 16;
    constexpr int kPieces = ROPE / 8;  // 16-byte pieces of a row's rotated part
    bool ok = true;
    int acc = 0;
    for (int u = unit0; u < units; u += step) {
      bool good;
      const int64_t page = page_of(u, good);
      const int entry = entry_of(u);
      if (!good && entry < a.entries && threadIdx.x == 0) atomicOr(a.err, kErrDeviceCheck);
      const int keys = good ? a.keys[entry] : 0;
      uint4 tail[kPieces];  // the same for every head
      if (which == 0) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int e = 32 * i + lane, r = row0 + e / kPieces;
          if (r < keys)
            tail[i] = *reinterpret_cast<const uint4*>(a.latent + (page * 128 + r) * a.width + a.chunks * 64 + e % kPieces * 8);
        }
      }
      for (int i = 0; i < heads_of(u); ++i, ++acc) {
        const int h = head_of(u, i);
        if (ok) ok = wait_cluster(d_full + (acc & 1), acc >> 1 & 1, a.err);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        const uint32_t at = tmem + (acc & 1) * 256 + lane_base + (which == 0 ? 0 : kNope);
        __nv_bfloat16* dst = (which == 0 ? a.k_pages : a.v_pages) + ((page * a.heads + h) * 128 + row0) * D;
        const int mine = ok ? keys - row0 : 0;  // of this warp's rows, those with keys
        auto columns = [&](auto n_cols) {
          constexpr int kCols = decltype(n_cols)::value;
#pragma unroll
          for (int c = 0; c + 32 <= kCols; c += 32)
#pragma unroll
            for (int half16 = 0; half16 < 2; ++half16) {
              uint32_t v[16], w[4];
              tmem_ld_16x256<4>(at + c + (static_cast<uint32_t>(half16 * 16) << 16), v);
              tmem_wait_ld();
#pragma unroll
              for (int q = 0; q < 2; ++q) {  // rows quad and quad + 8; a lane's two columns of each eight
#pragma unroll
                for (int g = 0; g < 4; ++g)
                  w[g] = pack_bf16x2(__uint_as_float(v[4 * g + 2 * q]), __uint_as_float(v[4 * g + 2 * q + 1]));
                transpose4(w, j);
                const int r = half16 * 16 + 8 * q + quad;
                if (r < mine) *reinterpret_cast<uint4*>(dst + r * D + c + 8 * j) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          if constexpr (kCols % 32 != 0) {
#pragma unroll
            for (int half16 = 0; half16 < 2; ++half16) {
              constexpr int c = kCols - 16;
              uint32_t v[8], w[4];
              tmem_ld_16x256<2>(at + c + (static_cast<uint32_t>(half16 * 16) << 16), v);
              tmem_wait_ld();
#pragma unroll
              for (int g = 0; g < 4; ++g)  // eight columns g & 1, rows quad + 8 (g >> 1)
                w[g] = pack_bf16x2(__uint_as_float(v[4 * (g & 1) + (g & 2)]), __uint_as_float(v[4 * (g & 1) + (g & 2) + 1]));
              transpose4(w, j);
              const int r = half16 * 16 + 8 * (j >> 1) + quad;
              if (r < mine) *reinterpret_cast<uint4*>(dst + r * D + c + 8 * (j & 1)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        };
        if (which == 0)
          columns(std::integral_constant<int, kNope>{});
        else
          columns(std::integral_constant<int, D>{});
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(d_empty + (acc & 1));
        if (which == 0)
#pragma unroll
          for (int k = 0; k < kPieces; ++k) {
            const int e = 32 * k + lane, r = e / kPieces;
            if (r < mine) *reinterpret_cast<uint4*>(dst + r * D + kNope + e % kPieces * 8) = tail[k];
          }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no product reads the other CTA's shared memory any more
  tc_fence_after();
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Heads a unit: the fewest rounds of the persistent grid, a unit's start
// counting as a head and a half.
int heads_per_unit(int64_t pairs, int heads, int clusters) {
  int best = heads;
  double least = 1e300;
  for (int groups = 1; groups <= heads; ++groups) {
    const int per = (heads + groups - 1) / groups;
    const int64_t units = pairs * ((heads + per - 1) / per);
    const double t = static_cast<double>((units + clusters - 1) / clusters) * (per + 1.5);
    if (t < least) least = t, best = per;
  }
  return best;
}

msa_status launch_expand(const msa_plan_s* p, const void* latent_pages, const void* w_k, const void* w_v,
                         const int32_t* kv_indices, int32_t latent_dim, int32_t rope_dim, void* k_pages, void* v_pages,
                         cudaStream_t st) {
  const int width = latent_dim + rope_dim, nope = p->d - rope_dim;
  const int half = product_cols(nope, p->d) / 2;
  CUtensorMap cm, km, v0, v1;
  auto rows = [](CUtensorMap* m, const void* base, int64_t n, int wide, int box_rows) {
    const uint64_t dims[2] = {static_cast<uint64_t>(wide), static_cast<uint64_t>(n)};
    const uint64_t str[1] = {static_cast<uint64_t>(wide) * 2};
    const uint32_t box[2] = {64, static_cast<uint32_t>(box_rows)};
    return encode_tensor_map(m, 2, base, dims, str, box, 1, 128);
  };
  if (!rows(&cm, latent_pages, p->num_pages * 128, width, 128) || !rows(&km, w_k, int64_t(p->hkv) * nope, latent_dim, nope) ||
      !rows(&v0, w_v, int64_t(p->hkv) * p->d, latent_dim, half - nope) ||
      !rows(&v1, w_v, int64_t(p->hkv) * p->d, latent_dim, nope + p->d - half))
    return set_error(MSA_ERR_CUDA, "msa_latent_expand: tensor map encoding failed");
  ExpandArgs a{};
  a.latent = static_cast<const __nv_bfloat16*>(latent_pages);
  a.kv_indices = kv_indices;
  a.keys = reinterpret_cast<const uint8_t*>(p->aux_d + p->entry_keys_off);
  a.k_pages = static_cast<__nv_bfloat16*>(k_pages);
  a.v_pages = static_cast<__nv_bfloat16*>(v_pages);
  a.err = p->err_d;
  a.num_pages = p->num_pages;
  a.entries = p->n_page_entries;
  a.heads = p->hkv;
  a.pairs = (a.entries + 1) / 2;
  a.per_unit = heads_per_unit(a.pairs, p->hkv, p->num_sms / 2);
  a.groups = (p->hkv + a.per_unit - 1) / a.per_unit;
  a.chunks = latent_dim / 64;
  a.width = width;
  a.stages = std::min(kMaxStages, kRing / (2 * half * 128));
  const int64_t units = int64_t(a.pairs) * a.groups;
  if (units > 0x7FFFFFFF) return set_error(MSA_ERR_UNSUPPORTED, "msa_latent_expand: too many pages");
  const bool wide = p->d == 128;
  const auto kern = rope_dim == 16   ? (wide ? expand_kernel<128, 16> : expand_kernel<64, 16>)
                    : rope_dim == 32 ? (wide ? expand_kernel<128, 32> : expand_kernel<64, 32>)
                    : rope_dim == 48 ? (wide ? expand_kernel<128, 48> : expand_kernel<64, 48>)
                                     : expand_kernel<128, 64>;
  const int smem = kSmem + 1024;
  // the devices that have each kernel's limit (the call takes about a microsecond)
  static std::atomic<uint64_t> devices[8];
  std::atomic<uint64_t>& have = devices[rope_dim / 16 * 2 - 1 - wide];
  const uint64_t bit = p->device < 64 ? uint64_t(1) << p->device : 0;
  cudaError_t e = cudaSuccess;
  if ((have.load(std::memory_order_acquire) & bit) == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) have.fetch_or(bit, std::memory_order_release);
  }
  if (e == cudaSuccess)
    e = launch_pdl_cluster(kern, dim3(static_cast<unsigned>(2 * std::min<int64_t>(units, p->num_sms / 2))), 2,
                           dim3(kThreads), smem, st, cm, km, v0, v1, a);
  return cuda_check(e, "msa_latent_expand: launch");
}

}  // namespace

// Keys of each page-table entry's page, a byte each: 128, and what is left in a sequence's
// last.  Every plan of bf16 has them, those of decode steps over long contexts too, so they
// are few bytes (32 sequences of 131072 keys: a plan takes 340 us with int32s, 302 with bytes,
// 284 without).
void expand_plan_tables(msa_plan_s* p, std::vector<int32_t>& aux) {
  if (p->kv_dtype != MSA_KV_BF16) return;
  p->entry_keys_off = static_cast<int64_t>(aux.size());
  static_assert(kPage == 128);
  aux.resize(aux.size() + (size_t(p->n_page_entries) + 3) / 4, static_cast<int32_t>(0x80808080u));
  uint8_t* end = reinterpret_cast<uint8_t*>(aux.data() + p->entry_keys_off);
  for (int32_t k : p->kv_lens) {
    end += (int64_t(k) + kPage - 1) / kPage;
    if (k % kPage != 0) end[-1] = static_cast<uint8_t>(k % kPage);
  }
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
