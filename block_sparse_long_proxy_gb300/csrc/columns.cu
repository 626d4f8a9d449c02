// Attention of few query rows over the paged caches: trees of drafted tokens
// over K/V pages (msa_tree_attn), and the absorbed form over a cache of one
// shared latent vector a token (msa_latent_attn).
//
// For query row i of tile t and head h of proxy head p, over the keys of the
// blocks kv_block_indexes[t, p, :] that i sees,
//   s = q[i,h] . k[key] * scale,  out = sum softmax(s) v[key],  lse = ln sum e^s.
// In the latent cache every head's key is [latent | rotated part] and its
// value the latent: one array, read once for both products.
//
// The heads of p (all of them, in the latent cache) share keys and values, so a
// tile of a few rows is already a matrix: its columns are the (row, head)
// pairs, column c being head c % G of row c / G.  Products are transposed,
//   S^T [128 keys x N] = K_block . Q^T         (M = 128 keys)
//   O^T [dims x N]    += V_block^T . P^T       (M = 128 dims a product)
// so that a block always fills the 128 M rows of tcgen05.mma, however few the
// columns, and N = 16..128 follows the batch.  (With the rows as M, eight heads
// of one row would fill 8 of 128.)  O^T of 64 columns and a 512-wide latent
// takes 256 TMEM columns, where 64 x 512 with the rows as M takes all 512.
//
// Roles: one warp lists the blocks and issues TMA loads into a ring of 32 KB slots
// (K or V of a block; 128 of the latent's dims); one issues the products; 8 or 16
// softmax warps, each four of them a share of the columns and a thread a key,
// mask, find each column's maximum, and write P^T (bf16, or f16 for e4m3 caches: a
// weight is off by 2^-8 or 2^-11 of itself at most, the sums being of the unrounded
// ones) back to shared memory.  The latent's P^T goes where the block's rotated part
// was, which no product reads after S^T.  e4m3: four more warps expand the codes
// to f16 (exact) inside the slot.
//
// Softmax in the log2 domain; a column's reference moves only when its maximum
// grows by more than 2^8, so O^T is rarely rescaled.  Sums stay with the thread
// that has the key, in fp32, and are added over the keys once, at the end.
//
// The block scales of MSA_KV_FP8_E4M3_BLOCK are a BlockScale (msa_internal.h);
// static scales are the same with one scale for all pages.
//
// Visibility: key offset e = key - pos0 (pos0: the tile's first position) is
// seen by all rows below 0, by none from 128 on, and by row i in between iff bit
// e of its 128-bit mask is set: the tree's, or bits 0..i (causal).  A key that
// no column sees has its V row zeroed in shared memory: its bytes may be
// anything, and 0 * NaN is NaN.
//
// Few tiles: the CTAs of a cluster take a part of the blocks each and merge O^T,
// m and l over distributed shared memory; no workspace, so calls may overlap.
//
// Measured out of HBM, 16 blocks a row:
//   32 trees of 8 rows, 64/8 heads, bf16 (277 MB): 50 us, 5.5 TB/s.  Bound by HBM.
//   32 trees of 64 rows, 64/8 heads, e4m3 (138 GFLOP of products): 137 us (rows_kernel
//     below; as columns 293), 1.0 PFLOP/s.  Bound by a tile's chain from S to the next S,
//     1.6 us of which the exponentials of both tiles are 1.07.
//   latent, a chunk of 512 rows x 32 heads, 512 + 64 (73 GFLOP): 106 us, 0.69 PFLOP/s.
//     Bound by shared memory: 575 KB a block and 64 columns, at 128 B/clk 4500 of
//     the 5400 clocks that a block takes.
//   latent decode, 32 sequences x 64 heads (80 MB): 28 us, 24 from the L2: a CTA has
//     4 blocks, and the merge of 4 parts moves 98 KB a CTA.
//   one tree of 16 rows: 12 us, one tile's chain of launch, tables, loads, products
//     and merge.
#include "msa_internal.h"
#include "ptx.cuh"

#include <algorithm>
#include <atomic>

namespace msa {
namespace {

enum Cache { kBf16, kE4m3, kLatent };

constexpr int kSlotBytes = 32768;
constexpr int kMaxParts = 16;

__device__ __forceinline__ float redux_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// Named barrier `id` over n threads that also returns the OR of p over them.
__device__ __forceinline__ bool bar_sync_or(int id, bool p, int n) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %1, 0;\n\t"
      "bar.red.or.pred b, %2, %3, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
  if constexpr (C == 8) tmem_ld8(taddr, r);
  if constexpr (C == 16) tmem_ld16(taddr, r);
  if constexpr (C == 32) tmem_ld32(taddr, r);
}
template <int C>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t* r) {
  if constexpr (C == 8) tmem_st8(taddr, r);
  if constexpr (C >= 16) tmem_st16(taddr, r);
  if constexpr (C == 32) tmem_st16(taddr + 16, r + 16);
}

// mma_ss, mma_ts and mma_commit by the lane that has `leader`
__device__ __forceinline__ void mma_ss_if(bool leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(leader))
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(bool leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(leader))
      : "memory");
}
__device__ __forceinline__ void mma_commit_if(bool leader, uint64_t* bar) {
  if (leader) mma_commit(bar);
}

struct ColArgs {
  const __nv_bfloat16* q;   // [total_q, hq, dq]
  const TileInfo* tiles;
  const int32_t* idx;
  const int32_t* kv_indices;
  const uint32_t* tree_mask;  // [total_q, 4]; nullptr: causal
  const float* k_scale;
  const float* v_scale;
  __nv_bfloat16* out;       // [total_q, hq, dv]
  float* lse;
  uint32_t* err;
  int64_t num_pages;
  int32_t hq, hp, hkv;
  int32_t topk, parts, max_groups;
  int32_t dq, dv;
  int32_t kc;               // 64-column chunks of a key
  int32_t mt;               // 128-row products of O^T
  int32_t per_page;         // e4m3: a scale for each (page, KV head)
  int32_t q_tma;            // bf16: Q^T by q_map
  float scale_log2;
};

// A tile of the plan, before pdl_wait: no kernel writes the plan's tables, and L2 has
// what msa_plan uploaded.
__device__ __forceinline__ TileInfo plan_tile(const TileInfo* at) {
  const int4 x = __ldcg(reinterpret_cast<const int4*>(at)), y = __ldcg(reinterpret_cast<const int4*>(at) + 1);
  return TileInfo{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}

// the bits of word k of a 128-bit mask that lie below n
__device__ __forceinline__ uint32_t low_bits(int k, int n) {
  return n >= 32 * (k + 1) ? 0xFFFFFFFFu : n <= 32 * k ? 0u : (1u << (n - 32 * k)) - 1u;
}

// A part's blocks, by one warp: padding skipped, what lies behind the tile's last
// block or on a page outside the pool dropped and reported.  list[]: page | place
// << 24, the place 0 for a block before the tile's first position, 1 for that
// position's, 2 for the next; scales[] as a BlockScale has them.  sel: the selection,
// j0 its first 32.  first(n) is called when those are listed.
template <bool FP8, class F>
__device__ __forceinline__ int list_blocks(const ColArgs& a, const TileInfo& tl, const int32_t* sel, int j0, int kvh,
                                           int part, int parts, uint32_t* list, float2* scales, F first32) {
  const int lane = threadIdx.x & 31;
  auto at = [&](int b) { return b == 0 ? j0 : b + lane < a.topk ? sel[b + lane] : -1; };
  int first = 0, count = a.topk, seen = 0, n = 0;
  if (parts > 1) {
    int total = 0;
    for (int b = 0; b < a.topk; b += 32) {
      const int j = at(b);
      total += __popc(__ballot_sync(0xFFFFFFFFu, j >= 0 && j < tl.nvp));
    }
    first = total * part / parts;
    count = total * (part + 1) / parts - first;
  }
  const int first_masked = tl.pos0 >> 7;
  for (int b = 0; b < a.topk; b += 32) {
    const int j = at(b);
    const bool valid = j >= 0 && j < tl.nvp;
    const uint32_t v = __ballot_sync(0xFFFFFFFFu, valid), below = (1u << lane) - 1u;
    const int rank = seen + __popc(v & below);
    seen += __popc(v);
    bool take = valid && rank >= first && rank < first + count, bad = j >= tl.nvp;
    int64_t page = 0;
    if (take) {
      page = a.kv_indices[tl.page_base + j];
      if (page < 0 || page >= a.num_pages) take = false, bad = true;
    }
    if (bad) atomicOr(a.err, kErrDeviceCheck);
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, take);
    const int o = n + __popc(m & below);
    if (take) list[o] = static_cast<uint32_t>(page) | static_cast<uint32_t>(max(j - first_masked + 1, 0)) << 24;
    n += __popc(m);
    __syncwarp();
    float ks = 0.f, vs = 0.f;  // on their way while the first loads are issued
    if (FP8 && take) {
      const int64_t sat = a.per_page ? page * a.hkv + kvh : kvh;
      ks = a.k_scale[sat], vs = a.v_scale[sat];
    }
    if (b == 0) first32(n);
    if (FP8 && take) {
      const BlockScale bs = block_scale_of(ks, vs);
      scales[o] = make_float2(bs.ks * a.scale_log2, bs.log2_vs);
    }
  }
  return n;
}

// e4m3: one key's codes of a slot (upper half) to its f16 row, zeros for `zero`.  A
// thread has the codes in registers before it writes that row, the only one that
// overlaps them (dims 128; at dims 64 none does).
__device__ __forceinline__ void expand_row(uint8_t* buf, int r, bool dims128, bool zero) {
  const int sw = r & 7;
  auto expand = [&](uint4 v, int unit) {  // sixteen codes -> f16 units 2 unit, 2 unit + 1
    if (zero) v = make_uint4(0u, 0u, 0u, 0u);
    uint8_t* dst = buf + (unit >> 2) * 16384 + r * 128;
    const int u0 = (unit & 3) * 2;
    *reinterpret_cast<uint4*>(dst + ((u0 ^ sw) << 4)) = make_uint4(
        e4m3x2_to_f16x2(v.x), e4m3x2_to_f16x2(v.x >> 16), e4m3x2_to_f16x2(v.y), e4m3x2_to_f16x2(v.y >> 16));
    *reinterpret_cast<uint4*>(dst + (((u0 + 1) ^ sw) << 4)) = make_uint4(
        e4m3x2_to_f16x2(v.z), e4m3x2_to_f16x2(v.z >> 16), e4m3x2_to_f16x2(v.w), e4m3x2_to_f16x2(v.w >> 16));
  };
  uint4 v[8];
  if (dims128) {
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = *reinterpret_cast<const uint4*>(buf + 16384 + r * 128 + ((c ^ sw) << 4));
#pragma unroll
    for (int c = 0; c < 8; ++c) expand(v[c], c);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = *reinterpret_cast<const uint4*>(buf + 16384 + r * 64 + ((c ^ (r >> 1 & 3)) << 4));
#pragma unroll
    for (int c = 0; c < 4; ++c) expand(v[c], c);
  }
}

template <int KIND, int N, bool TWO>
struct ColSmem {
  static constexpr bool kLat = KIND == kLatent;
  static constexpr int kQChunk = N * 128;
  static constexpr int kPBytes = kLat ? 0 : (N > 64 ? 32768 : 16384);
  static constexpr int kSlots = kLat ? (N == 64 ? 4 : 5) : TWO ? 2 : 4;
  static constexpr int kTails = kLat ? (N == 16 ? 2 : 1) : 0;  // slots of the rotated part, then P^T
  static constexpr int kTailBytes = 16384;
  static constexpr int kQOff = 0;
  static constexpr int kPOff = kQOff + (kLat ? 9 : 2) * kQChunk;
  static constexpr int kRingOff = kPOff + kPBytes;
  static constexpr int kTailOff = kRingOff + kSlots * kSlotBytes;
  static constexpr int kBarOff = kTailOff + kTails * kTailBytes;
  static constexpr int kMaskWords = N > 32 ? N / 32 : 1;
  static constexpr int kMaskOff = kBarOff + 8 * 32;        // [128 key offsets] the columns that see it
  static constexpr int kColOff = kMaskOff + 512 * kMaskWords;  // (m, l) of the columns
  static constexpr int kRedOff = kColOff + 8 * N;          // [warpgroup][4][columns] column maxima, or sums, of the warps
  static constexpr int kShiftOff = kRedOff + 16 * N;       // [warp][columns], twice: shift, rescaling factor
  static constexpr int kRowOff = kShiftOff + 2 * 16 * N;
  static constexpr int kListOff = kRowOff + 8 * N;
  static __host__ __device__ constexpr int bytes(int topk) {
    return kListOff + ((topk + 3) & ~3) * (KIND == kE4m3 ? 12 : 4);
  }
  static_assert(kQChunk % 1024 == 0 && kRingOff % 1024 == 0 && kTailOff % 1024 == 0, "swizzled tiles");
  // after the last block, a part's O^T: [N][dims] floats where the ring was (512 dims at most for
  // the latent cache, 128 for the others)
  static_assert(TWO || N * (kLat ? 512 : 128) * 4 <= kSlots * kSlotBytes, "O^T of a part fits the ring");
  // the weights of a merge, where Q was
  static_assert(N * kMaxParts * 4 <= kPOff, "weights fit Q's place");
};

// Softmax warpgroups: 8 to 32 columns each.  Alone on an SM, two of them leave the
// passes over S^T waiting for their own latencies; e4m3 of 32 columns rather has the
// registers for four more converter warps.
template <int KIND, int N, bool TWO>
constexpr int soft_warps() {
  return N == 16 || TWO || (KIND == kE4m3 && N == 32) ? 8 : 16;
}
// Converter warps, e4m3 only: four a slot; of eight, four have the K slots and four
// the V slots.
constexpr int kConvWarps = 4;
template <int KIND, int N>
constexpr int conv_warps() {
  return KIND != kE4m3 ? 0 : N <= 32 ? 8 : 4;
}
template <int KIND, int N, bool TWO>
constexpr int col_threads() {
  return 32 * (soft_warps<KIND, N, TWO>() + 2 + conv_warps<KIND, N>());
}

// Sums of CH values a lane over the warp's lanes: lane c (mod CH) has the sum of
// column c, in a fixed order.
template <int CH>
__device__ __forceinline__ float column_sums(float (&x)[CH], int lane) {
#pragma unroll
  for (int d = 16; d >= CH; d >>= 1)
#pragma unroll
    for (int j = 0; j < CH; ++j) x[j] += __shfl_xor_sync(0xFFFFFFFFu, x[j], d);
#pragma unroll
  for (int d = CH < 32 ? CH / 2 : 16; d > 0; d >>= 1)
#pragma unroll
    for (int j = 0; j < d; ++j) {
      const bool up = lane & d;
      const float send = up ? x[j] : x[j + d];
      x[j] = (up ? x[j + d] : x[j]) + __shfl_xor_sync(0xFFFFFFFFu, send, d);
    }
  return x[0];
}

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

template <int KIND, int N, bool TWO>
__global__ void __launch_bounds__(col_threads<KIND, N, TWO>(), TWO ? 2 : 1)
    columns_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                   const __grid_constant__ CUtensorMap q_map, const ColArgs a) {
  using L = ColSmem<KIND, N, TWO>;
  constexpr bool kLat = KIND == kLatent, kFp8 = KIND == kE4m3;
  constexpr int kThreads = col_threads<KIND, N, TWO>();
  constexpr int kSoftWarps = soft_warps<KIND, N, TWO>(), kProducer = kSoftWarps, kIssuer = kSoftWarps + 1;
  constexpr int kConv = conv_warps<KIND, N>();
  constexpr int HN = N / (kSoftWarps / 4);      // columns of a warpgroup
  constexpr int CH = 8;                         // of them, in registers at a time
  constexpr int NCH = HN / CH;
  constexpr bool kAhead = HN <= 16;
  constexpr int S = L::kSlots, T = L::kTails > 0 ? L::kTails : 1;
  constexpr uint32_t kTmemCols = kLat ? 8 * N : 4 * N;  // S^T twice, O^T of up to 4 products or 1
  constexpr float kUnset = 1e30f;  // minus the reference of a column that has none yet
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* full = bars;               // [S]: a slot's bytes (e4m3: codes) have landed
  uint64_t* empty = full + S;          // [S]
  uint64_t* ready = kFp8 ? empty + S : full;  // [S]: e4m3: expanded
  uint64_t* tail_full = empty + 2 * S;        // [kTails]
  uint64_t* tail_empty = tail_full + 2;
  uint64_t* s_full = tail_empty + 2;   // [2]
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 1;
  uint64_t* q_full = pv_done + 1;
  uint64_t* drain = q_full + 1;        // every product issued is complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int32_t* n_slot = reinterpret_cast<int32_t*>(tmem_slot + 1);
  uint32_t* seen_by = reinterpret_cast<uint32_t*>(smem + L::kMaskOff);
  float2* col_ml = reinterpret_cast<float2*>(smem + L::kColOff);
  int64_t* col_row = reinterpret_cast<int64_t*>(smem + L::kRowOff);  // (query row, head) of the columns, as a row of q and out
  uint32_t* list = reinterpret_cast<uint32_t*>(smem + L::kListOff);  // page | place of the block << 24
  float2* scales = reinterpret_cast<float2*>(list + ((a.topk + 3) & ~3));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = blockIdx.x % a.parts, unit = blockIdx.x / a.parts;
  const int group = unit % a.max_groups, p = unit / a.max_groups % a.hp, t = unit / a.max_groups / a.hp;
  const int G = a.hq / a.hp;
  const int kvh = p / (a.hp / a.hkv);

  // ------------------------------------------------------------- prologue
  if (warp == kProducer) {
    if (lane == 0) {
      prefetch_tmap(&k_map);
      prefetch_tmap(&v_map);
      for (int s = 0; s < S; ++s) {
        mbar_init(full + s, 1);
        mbar_init(empty + s, 1);
        if (kFp8) mbar_init(ready + s, kConvWarps);
      }
      for (int s = 0; s < 2; ++s) {
        mbar_init(tail_full + s, 1);
        mbar_init(tail_empty + s, 1);
        mbar_init(s_full + s, 1);
      }
      mbar_init(p_full, kSoftWarps);
      mbar_init(pv_done, 1);
      mbar_init(q_full, 1);
      mbar_init(drain, 1);
      fence_mbar_init();
    }
  } else if (warp == kIssuer) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  const TileInfo tl = plan_tile(a.tiles + t);
  pdl_wait();
  const int32_t* sel = a.idx + (static_cast<int64_t>(t) * a.hp + p) * a.topk;
  const int j0 = warp == kProducer && lane < a.topk ? sel[lane] : -1;
  const int c0 = group * N, cols = min(N, tl.rows * G - c0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Not before this CTA has its tensor memory: where it has to wait for that of another
  // stream's CTA, one of the next launch could take it first, and then waits for this one.
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  if (cols <= 0) {  // a tile of fewer rows than the batch's most (the whole cluster)
    if (warp == kIssuer) tmem_dealloc(tmem, kTmemCols);
    return;
  }
  const int per = kLat ? a.mt : 2;  // slot uses a block
  // slot uses so far -> slot and phase
  auto slot_of = [&](int u) { return u % S; };
  auto phase_of = [&](int u) { return static_cast<uint32_t>(u / S & 1); };
  // load h of block i: a slot, or (latent, h == per) the rotated part; by the whole
  // producer warp, `leader` issuing
  auto row_of = [&](int i) {
    return __shfl_sync(0xFFFFFFFFu, static_cast<int>((static_cast<int64_t>(list[i] & 0xFFFFFFu) * a.hkv + kvh) * 128), 0);
  };
  // the latent's next block on its way to L2: its slots are free only once this block's P.V is done
  auto prefetch = [&](int i, bool leader) {
    const int row = row_of(i);
    if (leader) {
      for (int h = 0; h < a.mt; ++h) tma_prefetch_3d(&v_map, 0, row, 2 * h);
      tma_prefetch_2d(&k_map, 128 * a.mt, row);
    }
  };
  int uses = 0, tails = 0;  // loads issued, to slots and of rotated parts
  auto produce = [&](int i, int h, bool leader) {
    const int row = row_of(i);
    auto waited = [&](uint64_t* bar, uint32_t parity) {
      return static_cast<bool>(__all_sync(0xFFFFFFFFu, mbar_wait_inl(bar, parity, a.err)));
    };
    if (kLat && h == per) {
      const int s = i % T;
      if (i >= T && !waited(tail_empty + s, (i / T & 1) ^ 1)) return false;
      if (leader) {
        mbar_expect_tx(tail_full + s, L::kTailBytes);
        tma_load_2d(smem + L::kTailOff + s * L::kTailBytes, &k_map, tail_full + s, 128 * a.mt, row);
      }
      tails = i + 1;
      return true;
    }
    const int u = i * per + h, s = slot_of(u);
    if (u >= S && !waited(empty + s, phase_of(u) ^ 1)) return false;
    uint8_t* dst = smem + L::kRingOff + s * kSlotBytes;
    if (leader) {
      if (kFp8) {
        mbar_expect_tx(full + s, 128 * a.dv);
        tma_load_2d(dst + 16384, h == 0 ? &k_map : &v_map, full + s, 0, row);
      } else if (kLat) {
        mbar_expect_tx(full + s, kSlotBytes);
        tma_load_3d(dst, &v_map, full + s, 0, row, 2 * h);
      } else {
        mbar_expect_tx(full + s, a.kc * 16384);
        tma_load_3d(dst, h == 0 ? &k_map : &v_map, full + s, 0, row, 0);
      }
    }
    uses = u + 1;
    return true;
  };
  // e4m3: slot use u's codes to f16, a thread a key, by four warps
  auto convert = [&](int u, bool zero) {
    const int s = slot_of(u);
    if (!__all_sync(0xFFFFFFFFu, mbar_wait_inl(full + s, phase_of(u), a.err))) return false;
    expand_row(smem + L::kRingOff + s * kSlotBytes, (threadIdx.x - 32 * (kIssuer + 1)) & 127, a.dv == 128, zero);
    fence_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(ready + s);
    return true;
  };
  bool conv_ok = true, converted = false;
  const int first_blocks = kLat ? 1 : S / 2;  // loaded before the columns are there
  int started = 0;
  if (warp == kProducer) {
    const int n = list_blocks<kFp8>(a, tl, sel, j0, kvh, part, a.parts, list, scales, [&](int n) {
      if (kFp8) {
        if (lane == 0) n_slot[1] = n;  // for the converters: is the first block among them?
        __syncwarp();
        asm volatile("bar.arrive 7, %0;" ::"n"(32 + 32 * kConv) : "memory");
      }
      started = min(n, first_blocks);
      const bool leader = elect_one();
      for (int i = 0; i < started; ++i)
        for (int h = 0; h < per + kLat; ++h) produce(i, h, leader);
    });
    if (lane == 0) *n_slot = n;
  } else if (kFp8 && warp > kIssuer) {
    // the first block's K, as soon as it has landed
    asm volatile("bar.sync 7, %0;" ::"n"(32 + 32 * kConv) : "memory");
    if (warp <= kIssuer + 4 && (converted = n_slot[1] > 0)) conv_ok = convert(0, false);
  } else {
    // Q^T's columns, 64 dims a chunk, a warp a column
    const int w = warp < kProducer ? warp : warp - 1;
    constexpr int kLoaders = kSoftWarps + 1;
    const uint32_t qs = smem_u32(smem + L::kQOff);
    const int units = a.kc * 8;
    if (kFp8) {
      // two or four columns a warp at once, converted on the way
      const int lg = a.kc == 2 ? 4 : 3;
      constexpr int kMost = (N * 16 + kLoaders * 32 - 1) / (kLoaders * 32);
      uint4 v[kMost];
#pragma unroll
      for (int k = 0; k < kMost; ++k) {
        const int e = (k * kLoaders + w) * 32 + lane, c = e >> lg, u = e & (units - 1);
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (c < cols)
          v[k] = *reinterpret_cast<const uint4*>(
              a.q + (static_cast<int64_t>(tl.q_begin + (c0 + c) / G) * a.hq + p * G + (c0 + c) % G) * a.dq + u * 8);
      }
#pragma unroll
      for (int k = 0; k < kMost; ++k) {
        const int e = (k * kLoaders + w) * 32 + lane, c = e >> lg, u = e & (units - 1);
        if (c < N)
          *reinterpret_cast<uint4*>(smem + L::kQOff + (u >> 3) * L::kQChunk + c * 128 + (((u & 7) ^ (c & 7)) << 4)) =
              make_uint4(bf16x2_to_f16x2(v[k].x), bf16x2_to_f16x2(v[k].y), bf16x2_to_f16x2(v[k].z), bf16x2_to_f16x2(v[k].w));
      }
    } else if (a.q_tma) {
      // what a box has beside the tile's columns (other rows' values) stays in its columns
      if (warp == kIssuer && elect_one()) {
        prefetch_tmap(&q_map);
        mbar_expect_tx(q_full, a.kc * L::kQChunk);
        for (int c = 0; c < a.kc; ++c)
          tma_load_3d(smem + L::kQOff + c * L::kQChunk, &q_map, q_full, 64 * c, p * G + c0 % G, tl.q_begin + c0 / G);
      }
      __syncwarp();
    } else {
      const int cl = c0 + w + lane * kLoaders;  // a lane finds one column's row (a division by G)
      const int64_t at_l = static_cast<int64_t>(tl.q_begin + cl / G) * a.hq + p * G + cl % G;
      for (int c = w, k = 0; c < N; c += kLoaders, ++k) {
        const int64_t row = __shfl_sync(0xFFFFFFFFu, at_l, k);
        const __nv_bfloat16* src = c < cols ? a.q + row * a.dq : a.q;
        for (int u = lane; u < units; u += 32) {
          const bool there = c < cols && u * 8 < a.dq;
          copy16_async(qs + (u >> 3) * L::kQChunk + c * 128 + (((u & 7) ^ (c & 7)) << 4), there ? src + u * 8 : a.q, there);
        }
      }
    }
    // what each column is, and sees
    const int th = w * 32 + lane;
    for (int c = th; c < N; c += kLoaders * 32)
      col_row[c] = static_cast<int64_t>(tl.q_begin + (c0 + c) / G) * a.hq + p * G + (c0 + c) % G;
    for (int e0 = w * 32; e0 < N * 4; e0 += kLoaders * 32) {
      const int e = e0 + lane, c = e % N, wd = e / N, row = (c0 + c) / G;
      uint32_t m = 0u;
      if (c < cols)
        m = a.tree_mask ? a.tree_mask[4 * static_cast<int64_t>(tl.q_begin + row) + wd] & low_bits(wd, tl.rows) : low_bits(wd, row + 1);
      // a row of bits a column -> a row a key offset; lane b keeps offset 32 wd + b
      uint32_t mine = 0u;
#pragma unroll
      for (int d = 0; d < 32; ++d) {
        const uint32_t w = __ballot_sync(0xFFFFFFFFu, m >> d & 1u);
        if (lane == d) mine = w;
      }
      if (N >= 32) {
        seen_by[(32 * (e0 / N) + lane) * L::kMaskWords + e0 % N / 32] = mine;
      } else {  // 16 columns of two words
        seen_by[64 * (e0 / 32) + lane] = mine & 0xFFFFu;
        seen_by[64 * (e0 / 32) + 32 + lane] = mine >> 16;
      }
    }
    if (!kFp8) asm volatile("cp.async.wait_all;" ::: "memory");
  }
  fence_async_shared();
  __syncthreads();
  const int n = *n_slot;
  // key offset of lane 0 of block i's rows; places: 0 before the tile, 1 its first block, 2 the next
  auto offset0 = [&](uint32_t entry) { return (static_cast<int>(entry >> 24) - 1) * 128 - (tl.pos0 & 127); };
  auto seen_by_any = [&](int e) {
    if (e < 0 || e >= 128) return e < 0;
    uint32_t any = 0u;
    for (int w = 0; w < L::kMaskWords; ++w) any |= seen_by[e * L::kMaskWords + w];
    return any != 0u;
  };

  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one();
    bool ok = true;
    if (kLat && started > 0 && started < n) {
      // all CTAs' first blocks come from HBM at once: the second ones wait (32 sequences 28.2 -> 27.3 us)
      ok = __all_sync(0xFFFFFFFFu, mbar_wait_inl(full + slot_of(per - 1), 0, a.err));
      if (ok) prefetch(started, leader);
    }
    for (int i = started; i < n && ok; ++i) {
      if (kLat && i + 1 < n) prefetch(i + 1, leader);
      for (int h = 0; h < per + kLat && ok; ++h) ok = produce(i, h, leader);
    }
    // Nothing is under way to this CTA's shared memory when it leaves, although a role that
    // gave up a wait leaves loads unused.
    for (int u = max(uses - S, 0); u < uses; ++u) mbar_wait_inl(full + slot_of(u), phase_of(u), a.err);
    for (int i = max(tails - T, 0); i < tails; ++i) mbar_wait_inl(tail_full + i % T, i / T & 1, a.err);
  } else if (warp == kIssuer) {
    // ----------------------------------------------------------------- MMA
    // The whole warp goes through the loop, one elected lane issuing: descriptors
    // are then the warp's, not a lane's, and need no move to uniform registers.
    {
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const int nn = __shfl_sync(0xFFFFFFFFu, n, 0);
      const bool leader = elect_one();
      auto waited = [&](uint64_t* bar, uint32_t parity) {
        return static_cast<bool>(__all_sync(0xFFFFFFFFu, mbar_wait_inl(bar, parity, a.err)));
      };
      constexpr uint32_t id_qk = kFp8 ? idesc_f16_f32(128, N, false, false) : idesc_bf16_f32(128, N, false, false);
      constexpr uint32_t id_pv = kFp8 ? idesc_f16_f32(128, N, true, true) : idesc_bf16_f32(128, N, true, true);
      const uint64_t kd0 = smem_desc(smem_u32(smem + L::kRingOff), 16, 1024, kSwizzle128);
      const uint64_t qd0 = smem_desc(smem_u32(smem + L::kQOff), 16, 1024, kSwizzle128);
      // V^T: 64 dims a chunk, the second 64 one chunk on; at dims 64 both halves of M are the one chunk
      const uint64_t vd0 = smem_desc(smem_u32(smem + L::kRingOff), a.dv == 64 ? 0 : 16384, 1024, kSwizzle128);
      const uint64_t td0 = smem_desc(smem_u32(smem + L::kTailOff), 16, 1024, kSwizzle128);
      const uint64_t pd0 = smem_desc(smem_u32(smem + (kLat ? L::kTailOff : L::kPOff)), 16384, 1024, kSwizzle128);
      bool ok = true;
      auto qk = [&](int i) {
        const uint32_t d = tm + (i & 1) * N;
        uint32_t acc = 0;
        for (int h = 0; h < (kLat ? a.mt : 1); ++h) {
          const int u = i * per + h, s = slot_of(u);
          if (!(ok = waited(ready + s, phase_of(u)))) return;
          tc_fence_after();
          const uint64_t kd = kd0 + s * (kSlotBytes >> 4), qd = qd0 + h * 2 * (L::kQChunk >> 4);
          for (int c = 0; c < (kLat ? 2 : a.kc); ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              mma_ss_if(leader, d, kd + ((c * 16384 + kk * 32) >> 4), qd + ((c * L::kQChunk + kk * 32) >> 4), id_qk, acc);
              acc = 1;
            }
          if (!kLat) mma_commit_if(leader, empty + s);
        }
        if (kLat) {
          const int s = i % T;
          if (!(ok = waited(tail_full + s, i / T & 1))) return;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_if(leader, d, td0 + ((s * L::kTailBytes + kk * 32) >> 4), qd0 + ((2 * a.mt * L::kQChunk + kk * 32) >> 4), id_qk, 1);
        }
        mma_commit_if(leader, s_full + (i & 1));
      };
      if (!kFp8 && a.q_tma) ok = waited(q_full, 0);
      if (nn > 0 && ok) qk(0);
      for (int i = 0; i < nn && ok; ++i) {
        // the latent's slots serve S^T of block i until its P.V: the next block's loads wait for that
        if (!kLat && i + 1 < nn) qk(i + 1);
        if (!ok || !(ok = waited(p_full, i & 1))) break;
        tc_fence_after();
        const uint64_t pd = pd0 + (kLat ? (i % T) * (L::kTailBytes >> 4) : 0);
        for (int h = 0; h < a.mt && ok; ++h) {
          const int u = kLat ? i * per + h : i * per + 1, s = slot_of(u);
          if (!kLat) {
            if (!(ok = waited(ready + s, phase_of(u)))) break;
            tc_fence_after();
          }
          const uint64_t vd = vd0 + s * (kSlotBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss_if(leader, tm + (2 + h) * N, vd + ((kk * 2048) >> 4), pd + ((kk * 2048) >> 4), id_pv, i > 0 || kk > 0);
          mma_commit_if(leader, empty + s);
        }
        if (kLat) mma_commit_if(leader, tail_empty + i % T);
        mma_commit_if(leader, pv_done);
        if (kLat && ok && i + 1 < nn) qk(i + 1);
      }
      mma_commit_if(leader, drain);  // nor a product, also after a wait that was given up
      waited(drain, 0);
    }
  } else if (warp < kSoftWarps) {
    // ------------------------------------------------------------- softmax
    // Every warp goes through all n blocks whatever its waits say (they are
    // skipped after one that gave up), so the warpgroup's barriers stay whole.
    const int wg = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    float* const red = reinterpret_cast<float*>(smem + L::kRedOff) + wg * 4 * HN;
    float* shift = reinterpret_cast<float*>(smem + L::kShiftOff) + warp * 2 * HN;  // minus the references
    float* alpha = shift + HN;
    auto group_sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); };
    const uint32_t o_addr = tmem + lane_base + 2 * N + wg * HN;
    float l[NCH][CH], m[NCH];  // sums of this thread's keys; references of columns CH k + lane
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      m[k] = -INFINITY;
#pragma unroll
      for (int c = 0; c < CH; ++c) l[k][c] = 0.f;
      if (lane < CH) shift[k * CH + lane] = kUnset;
    }
    __syncwarp();
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = mbar_wait_inl(bar, parity, a.err);
      ok = __all_sync(0xFFFFFFFFu, ok);
    };
    for (int i = 0; i < n; ++i) {
      wait(s_full + (i & 1), i >> 1 & 1);
      tc_fence_after();
      const uint32_t entry = list[i];
      const uint32_t s_addr = tmem + lane_base + (i & 1) * N + wg * HN;
      float sl2 = a.scale_log2, log2_vs = 0.f, inv_vs = 1.f;
      if (kFp8) {
        const float2 sc = scales[i];
        sl2 = sc.x, log2_vs = sc.y, inv_vs = ex2_approx(-sc.y);
      }
      const bool masked = entry >> 24 != 0;
      const int e = offset0(entry) + r;
      uint32_t vis = 0xFFFFFFFFu;  // this warpgroup's columns that see the key
      if (masked && e >= 0)
        vis = e < 128 ? seen_by[e * L::kMaskWords + wg * HN / 32] >> (wg * HN % 32) : 0u;
      uint32_t s[CH];
      auto load = [&](int k) {
        tmem_ld<CH>(s_addr + k * CH, s);
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int c = 0; c < CH; ++c)
            if (!(vis >> (k * CH + c) & 1u)) s[c] = __float_as_uint(-INFINITY);
        }
      };
      // logits of columns c and c + 1 of chunk k less their references, log2
      auto logits = [&](int k, int c, float2 sh, float& x0, float& x1) {
        ffma2v(x0, x1, __uint_as_float(s[c]), __uint_as_float(s[c + 1]), sl2, sl2, sh.x, sh.y);
      };
      // with the block's log2 of the value scale, which every column's logits have
      auto put_shift = [&] {
#pragma unroll
        for (int k = 0; k < NCH; ++k)
          if (lane < CH) shift[k * CH + lane] = (m[k] == -INFINITY ? kUnset : -m[k]) + log2_vs;
        __syncwarp();
      };
      if (kFp8) put_shift();
      // P^T of chunk k by the present references, the sums that go with it, and the largest logit
      uint32_t w[kAhead ? NCH : 1][4];
      float far = -INFINITY;
      auto weigh = [&](int k, uint32_t (&w)[4], float (&l)[CH]) {
#pragma unroll
        for (int c = 0; c < CH; c += 4) {
          const float4 sh = *reinterpret_cast<const float4*>(shift + k * CH + c);
#pragma unroll
          for (int b = 0; b < 4; b += 2) {
            float x0, x1;
            logits(k, c + b, b == 0 ? make_float2(sh.x, sh.y) : make_float2(sh.z, sh.w), x0, x1);
            far = fmax3(far, x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            if (kFp8)
              ffma2v(l[c + b], l[c + b + 1], p0, p1, inv_vs, inv_vs, l[c + b], l[c + b + 1]);
            else
              fadd2(l[c + b], l[c + b + 1], p0, p1);
            w[(c + b) / 2] = kFp8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          }
        }
      };
      // does any column outgrow its reference?  (one without has kUnset, which any logit outgrows.)  With
      // few columns a warpgroup, P^T is there when the vote is; when it is lost, it is made again.
      float l_ahead[kAhead ? NCH : 1][CH];
      bool grown = i == 0;
      if (i > 0) {
        if constexpr (kAhead) {
#pragma unroll
          for (int k = 0; k < NCH; ++k) {
            load(k);
#pragma unroll
            for (int c = 0; c < CH; ++c) l_ahead[k][c] = l[k][c];
            weigh(k, w[k], l_ahead[k]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < NCH; ++k) {
            load(k);
#pragma unroll
            for (int c = 0; c < CH; c += 4) {
              const float4 sh = *reinterpret_cast<const float4*>(shift + k * CH + c);
              float x0, x1, x2, x3;
              logits(k, c, make_float2(sh.x, sh.y), x0, x1);
              logits(k, c + 2, make_float2(sh.z, sh.w), x2, x3);
              far = fmax3(fmax3(far, x0, x1), x2, x3);
            }
          }
        }
        grown = bar_sync_or(1 + wg, far > 8.f, 128);
      }
      if (grown) {
#pragma unroll
        for (int k = 0; k < NCH; ++k) {
          load(k);
          __syncwarp();
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const float x = redux_max(__uint_as_float(s[c]));
            if (lane == c) mx = x;
          }
          if (lane < CH) red[quarter * HN + k * CH + lane] = mx;
        }
        group_sync();
#pragma unroll
        for (int k = 0; k < NCH; ++k)
          if (lane < CH) {
            const int c = k * CH + lane;
            const float mx = fmaxf(fmaxf(red[c], red[HN + c]), fmaxf(red[2 * HN + c], red[3 * HN + c]));
            const float t2 = kFp8 ? fmaf(mx, sl2, log2_vs) : mx * sl2;
            const float m_new = t2 > m[k] + 8.f ? t2 : m[k];
            alpha[c] = m_new == m[k] ? 1.f : ex2_approx(m[k] - m_new);
            m[k] = m_new;
          }
        put_shift();
        if (i > 0) {  // O^T whole, then rescaled
          wait(pv_done, (i - 1) & 1);
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < NCH; ++k)
#pragma unroll
            for (int c = 0; c < CH; ++c) l[k][c] *= alpha[k * CH + c];
          for (int h = 0; h < a.mt; ++h)
#pragma unroll 1
            for (int k = 0; k < NCH; ++k) {
              uint32_t o[CH];
              tmem_ld<CH>(o_addr + h * N + k * CH, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < CH; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha[k * CH + c]);
              tmem_st<CH>(o_addr + h * N + k * CH, o);
            }
          tmem_wait_st();
        }
      }
      if (i > 0 && !kLat) wait(pv_done, (i - 1) & 1);  // P^T has one place
      uint8_t* pt = smem + (kLat ? L::kTailOff + (i % T) * L::kTailBytes : L::kPOff);
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        auto& wk = w[kAhead ? k : 0];
        if (!kAhead || grown) {
          if (NCH > 1) load(k);
          weigh(k, wk, l[k]);
        } else {
#pragma unroll
          for (int c = 0; c < CH; ++c) l[k][c] = l_ahead[kAhead ? k : 0][c];
        }
        const int col = wg * HN + k * CH;
        *reinterpret_cast<uint4*>(pt + (col >> 6) * 16384 + r * 128 + (((col >> 3 & 7) ^ (r & 7)) << 4)) =
            make_uint4(wk[0], wk[1], wk[2], wk[3]);
      }
      if (!kFp8 && masked) {  // V rows that no column sees (e4m3: the converters), 64 dims a warpgroup in turn
        if (!kLat) wait(full + slot_of(2 * i + 1), phase_of(2 * i + 1));
        if (!seen_by_any(e))
          for (int c = wg; c < (kLat ? 2 * a.mt : a.kc); c += kSoftWarps / 4) {
            uint8_t* v = smem + L::kRingOff + slot_of(kLat ? i * per + (c >> 1) : 2 * i + 1) * kSlotBytes + (c & 1) * 16384;
#pragma unroll
            for (int b = 0; b < 8; ++b) *reinterpret_cast<uint4*>(v + r * 128 + ((b ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
      }
      fence_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
    }

    // ------------------------------------------------------------ epilogue
    group_sync();  // red is free
    float total[NCH];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      total[k] = column_sums<CH>(l[k], lane);
      if (lane < CH) red[quarter * HN + k * CH + lane] = total[k];
    }
    group_sync();
#pragma unroll
    for (int k = 0; k < NCH; ++k)
      if (lane < CH) {
        const int c = k * CH + lane;
        total[k] = (red[c] + red[HN + c]) + (red[2 * HN + c] + red[3 * HN + c]);
        alpha[c] = total[k] > 0.f ? 1.f / total[k] : 0.f;
        if (quarter == 0) {
          col_ml[wg * HN + c] = make_float2(ok ? m[k] : -INFINITY, total[k]);
          if (a.parts == 1 && a.lse != nullptr && wg * HN + c < cols)
            a.lse[col_row[wg * HN + c]] = total[k] > 0.f ? (m[k] + log2f(total[k])) * 0.69314718055994531f : -INFINITY;
        }
      }
    __syncwarp();
    if (n > 0) wait(pv_done, (n - 1) & 1);
    tc_fence_after();
    float* part_o = reinterpret_cast<float*>(smem + L::kRingOff);
    for (int h = 0; h < a.mt; ++h)
#pragma unroll 1
      for (int k = 0; k < NCH; ++k) {
        uint32_t o[CH];
        if (n > 0) {
          tmem_ld<CH>(o_addr + h * N + k * CH, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int c = 0; c < CH; ++c) o[c] = 0u;
        }
        if (h * 128 + r >= a.dv) continue;  // dims 64: the upper half repeats the lower
        const int col0 = wg * HN + k * CH;
        if (!TWO && a.parts > 1) {
          float* to = part_o + col0 * a.dv + h * 128 + r;
#pragma unroll
          for (int c = 0; c < CH; ++c, to += a.dv) *to = __uint_as_float(o[c]);
          continue;
        }
        // even lanes take two dims of column c, odd lanes of column c + 1
        const bool odd = lane & 1;
        __nv_bfloat16* to = a.out + h * 128 + (r & ~1);
#pragma unroll
        for (int c = 0; c < CH; c += 2) {
          const float2 inv = *reinterpret_cast<const float2*>(alpha + k * CH + c);
          const float v0 = __uint_as_float(o[c]) * inv.x, v1 = __uint_as_float(o[c + 1]) * inv.y;
          const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v0 : v1, 1);
          if (col0 + c + odd < cols)
            *reinterpret_cast<uint32_t*>(to + col_row[col0 + c + odd] * a.dv) = odd ? pack_bf16x2(other, v1) : pack_bf16x2(v0, other);
        }
      }
  } else if (kFp8) {
    // ---------------------------------------------------------- converters
    const int r = (threadIdx.x - 32 * (kIssuer + 1)) & 127;
    const bool second = warp > kIssuer + 4;
    constexpr int kStride = kConv == 4 ? 1 : 2;
    for (int u = second ? 1 : converted ? kStride : 0; u < 2 * n && conv_ok; u += kStride) {
      const uint32_t entry = list[u >> 1];
      conv_ok = convert(u, (u & 1) && entry >> 24 != 0 && !seen_by_any(offset0(entry) + r));
    }
  }

  // ------------------------------------------------------------------- end
  tc_fence_before();
  if (TWO || a.parts == 1) {
    __syncthreads();
    tc_fence_after();
    if (warp == kIssuer) tmem_dealloc(tmem, kTmemCols);
    return;
  }
  cluster_sync();  // every part's O^T, m and l are in its shared memory
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, kTmemCols);
  // A share of the items each, four dims of one column.  Of more than four parts a
  // thread reads four and its neighbours the others, from this CTA's own on (all CTAs
  // reading one part's at a time took 1.5 times as long).  The first items are on
  // their way while the weights are made.
  float* wts = reinterpret_cast<float*>(smem + L::kQOff);  // [column][part]
  const int lg_parts = 31 - __clz(a.parts), lg_by = max(lg_parts - 2, 0), mine = a.parts >> lg_by;
  const int dv4 = a.dv / 4, items = cols * dv4;
  const int first = items * part / a.parts, last = items * (part + 1) / a.parts;
  const uint32_t ring = smem_u32(smem + L::kRingOff);
  const int by = threadIdx.x & ((1 << lg_by) - 1);
  float4 v[4];
  auto from = [&](int k) { return (part + by * mine + k) & (a.parts - 1); };
  auto fetch = [&](int e) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < mine) v[k] = ld_cluster_f4(ring + 16u * e, from(k));
  };
  float2 ml = make_float2(-INFINITY, 0.f);  // of the first columns: a thread one part's
  const int c_first = threadIdx.x >> lg_parts, w = threadIdx.x & (a.parts - 1);
  if (c_first < cols) ml = ld_cluster_f2(smem_u32(col_ml + c_first), w);
  int e = first + (threadIdx.x >> lg_by);
  if (e < last) fetch(e);
  for (int c = c_first; c - c_first < cols; c += kThreads >> lg_parts) {  // (all lanes of a warp alike)
    if (c != c_first) ml = c < cols ? ld_cluster_f2(smem_u32(col_ml + c), w) : make_float2(-INFINITY, 0.f);
    float mm = ml.x;
    for (int d = 1; d < a.parts; d *= 2) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, d));
    const float scale = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - mm);
    float sum = ml.y * scale;
    for (int d = 1; d < a.parts; d *= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    if (c < cols) {
      wts[c * kMaxParts + w] = sum > 0.f ? scale / sum : 0.f;
      if (part == 0 && w == 0 && a.lse != nullptr)
        a.lse[col_row[c]] = sum > 0.f ? (mm + log2f(sum)) * 0.69314718055994531f : -INFINITY;
    }
  }
  __syncthreads();
  // whole warps go round, as the parts' sums are added over neighbours
  for (int e0 = first + ((threadIdx.x & ~31) >> lg_by); e0 < last; e0 += kThreads >> lg_by) {
    const int c = e / dv4;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (e < last) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < mine) {
          const float x = wts[c * kMaxParts + from(k)];
          o.x += v[k].x * x, o.y += v[k].y * x, o.z += v[k].z * x, o.w += v[k].w * x;
        }
    }
    const int at = e;
    e += kThreads >> lg_by;
    if (e < last) fetch(e);
    for (int d = 1; d < 1 << lg_by; d *= 2) {
      o.x += __shfl_xor_sync(0xFFFFFFFFu, o.x, d), o.y += __shfl_xor_sync(0xFFFFFFFFu, o.y, d);
      o.z += __shfl_xor_sync(0xFFFFFFFFu, o.z, d), o.w += __shfl_xor_sync(0xFFFFFFFFu, o.w, d);
    }
    if (by == 0 && at < last)
      *reinterpret_cast<uint2*>(a.out + col_row[c] * a.dv + 4 * (at % dv4)) =
          make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  }
  cluster_sync();  // nobody leaves while its part may be read
}

// Wide trees: the (row, head) pairs as the M rows of the products, 128 to a tile and
// two tiles a CTA, as the prefill kernel has them,
//   S [128 pairs x 128 keys] = Q . K^T,   O [128 pairs x dims] += P . V,
// P in tensor memory where S was.  A thread has half a row of S, 64 keys, and its
// half of the sum until the end; the row's reference moves, as a column's does, only
// when some logit outgrows it by 2^8, which the tile's eight warps vote on, and
// only then do the halves exchange their maxima.  A block step serves 256 pairs.
// Both tiles share every K and V block, and one tile's softmax overlaps the other's
// products.
constexpr int kRowSoftWarps = 16;

template <bool FP8, int D>
struct RowSmem {
  static constexpr int kSlots = 4;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kRingOff = 2 * kTileBytes;
  static constexpr int kBarOff = kRingOff + kSlots * kSlotBytes;
  static constexpr int kAnyOff = kBarOff + 8 * 32;   // keys that some pair sees, by offset: 128 bits
  static constexpr int kRowOff = kAnyOff + 16;       // the pairs as rows of q and out
  static constexpr int kHalfOff = kRowOff + 8 * 256; // [tile][half][128] the halves' maxima, then sums
  static constexpr int kListOff = kHalfOff + 4 * 512;
  static __host__ __device__ constexpr int bytes(int topk) { return kListOff + ((topk + 3) & ~3) * (FP8 ? 12 : 4); }
};
template <bool FP8>
constexpr int row_threads() {
  return 32 * (kRowSoftWarps + 2 + (FP8 ? kConvWarps : 0));
}

template <bool FP8, int D>
__global__ void __launch_bounds__(row_threads<FP8>(), 1)
    rows_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const ColArgs a) {
  using L = RowSmem<FP8, D>;
  constexpr int kThreads = row_threads<FP8>(), S = L::kSlots, kProducer = kRowSoftWarps, kIssuer = kRowSoftWarps + 1;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);  // [S]
  uint64_t* empty = full + S;               // [S]
  uint64_t* ready = FP8 ? empty + S : full;  // [S]
  uint64_t* s_full = empty + 2 * S;         // [2 tiles]
  uint64_t* p_full = s_full + 2;            // [2]
  uint64_t* o_done = p_full + 2;            // [2] the last P.V
  uint64_t* drain = o_done + 2;             // every product issued is complete
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int32_t* n_slot = reinterpret_cast<int32_t*>(tmem_slot + 1);
  uint32_t* any = reinterpret_cast<uint32_t*>(smem + L::kAnyOff);
  int64_t* row_at = reinterpret_cast<int64_t*>(smem + L::kRowOff);
  uint32_t* list = reinterpret_cast<uint32_t*>(smem + L::kListOff);
  float2* scales = reinterpret_cast<float2*>(list + ((a.topk + 3) & ~3));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x % a.max_groups, p = blockIdx.x / a.max_groups % a.hp, t = blockIdx.x / a.max_groups / a.hp;
  const int G = a.hq / a.hp, kvh = p / (a.hp / a.hkv);
  if (warp == kProducer) {
    if (lane == 0) {
      prefetch_tmap(&k_map);
      prefetch_tmap(&v_map);
      for (int s = 0; s < S; ++s) {
        mbar_init(full + s, 1);
        mbar_init(empty + s, 1);
        if (FP8) mbar_init(ready + s, kConvWarps);
      }
      for (int h = 0; h < 2; ++h) {
        mbar_init(s_full + h, 1);
        mbar_init(p_full + h, 8);
        mbar_init(o_done + h, 1);
      }
      mbar_init(drain, 1);
      fence_mbar_init();
    }
    if (lane < 4) any[lane] = 0u;
  } else if (warp == kIssuer) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  const TileInfo tl = plan_tile(a.tiles + t);
  pdl_wait();
  const int32_t* sel = a.idx + (static_cast<int64_t>(t) * a.hp + p) * a.topk;
  const int j0 = warp == kProducer && lane < a.topk ? sel[lane] : -1;
  const int c0 = group * 256, pairs = min(256, tl.rows * G - c0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // (as in columns_kernel)
  const uint32_t tmem = *tmem_slot;
  if (pairs <= 0) {  // a tile of fewer rows than the batch's most
    if (warp == kIssuer) tmem_dealloc(tmem, 512);
    return;
  }
  const int tiles = pairs > 128 ? 2 : 1;
  auto slot_of = [&](int u) { return u % S; };
  auto phase_of = [&](int u) { return static_cast<uint32_t>(u / S & 1); };
  auto produce = [&](int u, bool leader) {  // K (u even) or V of block u / 2
    const int s = slot_of(u);
    const int row = __shfl_sync(
        0xFFFFFFFFu, static_cast<int>((static_cast<int64_t>(list[u >> 1] & 0xFFFFFFu) * a.hkv + kvh) * 128), 0);
    if (u >= S && !__all_sync(0xFFFFFFFFu, mbar_wait_inl(empty + s, phase_of(u) ^ 1, a.err))) return false;
    uint8_t* dst = smem + L::kRingOff + s * kSlotBytes;
    const CUtensorMap* map = u & 1 ? &v_map : &k_map;
    if (leader) {
      mbar_expect_tx(full + s, 128 * D * (FP8 ? 1 : 2));
      if (FP8)
        tma_load_2d(dst + 16384, map, full + s, 0, row);
      else
        tma_load_3d(dst, map, full + s, 0, row, 0);
    }
    return true;
  };
  int started = 0;
  if (warp == kProducer) {
    const int n = list_blocks<FP8>(a, tl, sel, j0, kvh, 0, 1, list, scales, [&](int n) {
      started = min(2 * n, S);
      const bool leader = elect_one();
      for (int u = 0; u < started; ++u) produce(u, leader);
    });
    if (lane == 0) *n_slot = n;
  } else {
    const int w = warp < kProducer ? warp : warp - 1;
    constexpr int kLoaders = kThreads / 32 - 1, kUnits = D / 8;
    if (w < 16) {  // Q, 16 pairs a warp: a lane finds one pair's row (a division by G), all load it
      const int c1 = c0 + 16 * w + (lane & 15);
      const int64_t row = static_cast<int64_t>(tl.q_begin + c1 / G) * a.hq + p * G + c1 % G;
      constexpr int kAtOnce = 32 / kUnits, kIters = 16 / kAtOnce;  // pairs a pass, passes
      const int u = lane % kUnits;
      uint8_t* dst = smem + (w >> 3) * L::kTileBytes + (u >> 3) * 16384;
      uint4 v[kIters];
#pragma unroll
      for (int k = 0; k < kIters; ++k) {
        const int j = k * kAtOnce + lane / kUnits;
        const int64_t from = __shfl_sync(0xFFFFFFFFu, row, j);
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (16 * w + j < pairs) v[k] = *reinterpret_cast<const uint4*>(a.q + from * D + u * 8);
      }
#pragma unroll
      for (int k = 0; k < kIters; ++k) {
        const int c = 16 * (w & 7) + k * kAtOnce + lane / kUnits;
        if (FP8)
          v[k] = make_uint4(bf16x2_to_f16x2(v[k].x), bf16x2_to_f16x2(v[k].y), bf16x2_to_f16x2(v[k].z), bf16x2_to_f16x2(v[k].w));
        *reinterpret_cast<uint4*>(dst + c * 128 + (((u & 7) ^ (c & 7)) << 4)) = v[k];
      }
    }
    for (int e = w * 32 + lane; e < 256; e += kLoaders * 32) {
      const int row = (c0 + e) / G;
      row_at[e] = static_cast<int64_t>(tl.q_begin + row) * a.hq + p * G + (c0 + e) % G;
      uint32_t x[4] = {0u, 0u, 0u, 0u};
      if (e < pairs) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[k] = a.tree_mask[4 * static_cast<int64_t>(tl.q_begin + row) + k] & low_bits(k, tl.rows);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t all = __reduce_or_sync(0xFFFFFFFFu, x[k]);
        if (lane == 0 && all != 0u) atomicOr(any + k, all);
      }
    }
  }
  fence_async_shared();
  __syncthreads();
  const int n = *n_slot;
  auto offset0 = [&](uint32_t entry) { return (static_cast<int>(entry >> 24) - 1) * 128 - (tl.pos0 & 127); };
  auto seen_by_any = [&](int e) { return e < 0 || (e < 128 && (any[e >> 5] >> (e & 31) & 1u)); };

  if (warp == kProducer) {
    const bool leader = elect_one();
    int uses = started;
    while (uses < 2 * n && produce(uses, leader)) ++uses;
    for (int u = max(uses - S, 0); u < uses; ++u)  // (as in columns_kernel)
      mbar_wait_inl(full + slot_of(u), phase_of(u), a.err);
  } else if (warp == kIssuer) {
    // ----------------------------------------------------------------- MMA
    // QK0 QK1 | PV0 QK0' PV1 QK1' | ...: one tile's softmax overlaps the other's products
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const int nn = __shfl_sync(0xFFFFFFFFu, n, 0);
    const bool leader = elect_one();
    auto waited = [&](uint64_t* bar, uint32_t parity) {
      return static_cast<bool>(__all_sync(0xFFFFFFFFu, mbar_wait_inl(bar, parity, a.err)));
    };
    constexpr uint32_t id_qk = FP8 ? idesc_f16_f32(128, 128, false, false) : idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t id_pv = FP8 ? idesc_f16_f32(128, D, false, true) : idesc_bf16_f32(128, D, false, true);
    const uint64_t qd0 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128);
    const uint64_t kd0 = smem_desc(smem_u32(smem + L::kRingOff), 16, 1024, kSwizzle128);
    const uint64_t vd0 = smem_desc(smem_u32(smem + L::kRingOff), 16384, 1024, kSwizzle128);
    auto qk = [&](int h, int s) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
        mma_ss_if(leader, tm + h * 128, qd0 + h * (L::kTileBytes >> 4) + off, kd0 + s * (kSlotBytes >> 4) + off, id_qk, kk > 0);
      }
      mma_commit_if(leader, s_full + h);
    };
    bool ok = nn == 0 || waited(ready, 0);
    tc_fence_after();
    if (ok && nn > 0) {
      qk(0, 0);
      if (tiles == 2) qk(1, 0);
      mma_commit_if(leader, empty);
    }
    for (int i = 0; i < nn && ok; ++i) {
      const int uv = 2 * i + 1, sv = slot_of(uv), sk = slot_of(uv + 1);
      if (!(ok = waited(ready + sv, phase_of(uv)))) break;
      for (int h = 0; h < tiles && ok; ++h) {
        if (!(ok = waited(p_full + h, i & 1))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_if(leader, tm + 256 + h * D, tm + h * 128 + kk / 4 * 64 + kk % 4 * 8, vd0 + sv * (kSlotBytes >> 4) + ((kk * 2048) >> 4), id_pv,
                    i > 0 || kk > 0);
        if (h == tiles - 1) mma_commit_if(leader, empty + sv);
        if (i + 1 < nn) {
          if (h == 0) {
            if (!(ok = waited(ready + sk, phase_of(uv + 1)))) break;
            tc_fence_after();
          }
          qk(h, sk);
          if (h == tiles - 1) mma_commit_if(leader, empty + sk);
        } else {
          mma_commit_if(leader, o_done + h);
        }
      }
    }
    mma_commit_if(leader, drain);
    waited(drain, 0);
  } else if (warp < kRowSoftWarps) {
    // ------------------------------------------------------------- softmax
    // tile, half of the keys, pair; every warp of a tile goes through all n blocks
    // whatever its waits say, so that the votes stay whole
    const int h = warp >> 3, half = warp >> 2 & 1, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + h * 128 + half * 64;
    const uint32_t o_addr = tmem + lane_base + 256 + h * D + half * (D / 2);
    const bool there = h * 128 + r < pairs;
    float* const halves = reinterpret_cast<float*>(smem + L::kHalfOff) + h * 256;
    auto tile_sync = [&] { asm volatile("bar.sync %0, 256;" ::"r"(1 + h) : "memory"); };
    uint32_t mask[4] = {0u, 0u, 0u, 0u};
    if (there) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mask[k] = a.tree_mask[4 * static_cast<int64_t>(tl.q_begin + (c0 + h * 128 + r) / G) + k] & low_bits(k, tl.rows);
    }
    // bits e .. e + 31 of: ones below 0, the mask, zeros from 128 on
    auto seen = [&](int e) {
      const int k = e >> 5;
      auto word = [&](int i) { return i < 0 ? 0xFFFFFFFFu : i == 0 ? mask[0] : i == 1 ? mask[1] : i == 2 ? mask[2] : i == 3 ? mask[3] : 0u; };
      return __funnelshift_r(word(k), word(k + 1), e & 31);
    };
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const int blocks = h < tiles ? n : 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = mbar_wait_inl(bar, parity, a.err);
      ok = __all_sync(0xFFFFFFFFu, ok);
    };
    for (int i = 0; i < blocks; ++i) {
      const uint32_t entry = list[i];
      float sl2 = a.scale_log2, log2_vs = 0.f, inv_vs = 1.f;
      if (FP8) {
        const float2 sc = scales[i];
        sl2 = sc.x, log2_vs = sc.y, inv_vs = ex2_approx(-sc.y);
      }
      const bool masked = entry >> 24 != 0;
      const int e0 = offset0(entry);
      uint32_t vis[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
      if (masked) vis[0] = seen(e0 + half * 64), vis[1] = seen(e0 + half * 64 + 32);
      wait(s_full + h, i & 1);
      tc_fence_after();
      uint32_t s[16];
      auto load = [&](int c) {
        tmem_ld16(s_addr + 16 * c, s);
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (!(vis[c >> 1] >> (16 * (c & 1) + k) & 1u)) s[k] = __float_as_uint(-INFINITY);
        }
      };
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t x[32];
        tmem_ld32(s_addr + 32 * c, x);
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!(vis[c] >> k & 1u)) x[k] = __float_as_uint(-INFINITY);
        }
#pragma unroll
        for (int k = 0; k < 32; k += 2) mx = fmax3(mx, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
      }
      const float mx2 = FP8 ? fmaf(mx, sl2, log2_vs) : mx * sl2;
      if (bar_sync_or(1 + h, mx2 > m + 8.f, 256)) {  // m is -inf at first
        halves[half * 128 + r] = mx2;
        tile_sync();
        const float both = fmaxf(mx2, halves[(half ^ 1) * 128 + r]);
        const float m_new = both > m + 8.f ? both : m;
        const float alpha = m_new == m ? 1.f : ex2_approx(m - m_new);
        l *= alpha;
        m = m_new;
        // P.V of the block before is complete: this block's S was issued after it
        if (i > 0 && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {  // this half's dims
            uint32_t o[16];
            tmem_ld16(o_addr + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st16(o_addr + 16 * c, o);
          }
        }
      }
      const float shift = log2_vs - (m == -INFINITY ? 0.f : m);
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        load(c);
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float x0, x1;
          ffma2(x0, x1, __uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1]), sl2, shift);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          fadd2(sum0, sum1, p0, p1);
          w[k] = FP8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
        }
        tmem_st8(s_addr + 8 * c, w);  // over keys of this half that are read
      }
      l += FP8 ? (sum0 + sum1) * inv_vs : sum0 + sum1;
      if (!FP8 && masked && h == 0) {  // V rows that no pair sees (e4m3: the converters), 64 dims a half
        wait(full + slot_of(2 * i + 1), phase_of(2 * i + 1));
        if (!seen_by_any(e0 + r) && half < D / 64) {
          uint8_t* v = smem + L::kRingOff + slot_of(2 * i + 1) * kSlotBytes + half * 16384 + r * 128;
#pragma unroll
          for (int b = 0; b < 8; ++b) *reinterpret_cast<uint4*>(v + ((b ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_shared();
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + h);
    }

    // ------------------------------------------------------------ epilogue
    if (h < tiles) {
      tile_sync();  // halves is free
      halves[half * 128 + r] = l;
      tile_sync();
      l = halves[r] + halves[128 + r];
      if (n > 0) wait(o_done + h, 0);
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      if (there && ok && half == 0 && a.lse != nullptr)
        a.lse[row_at[h * 128 + r]] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      const int quad = lane >> 2, j = lane & 3;
#pragma unroll
      for (int half16 = 0; half16 < 2; ++half16) {
        float iv[2];
        __nv_bfloat16* dst[2];
        bool mine[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int rr = half16 * 16 + 8 * q + quad, pair = h * 128 + quarter * 32 + rr;
          iv[q] = __shfl_sync(0xFFFFFFFFu, inv, rr);
          mine[q] = pair < pairs && ok;
          dst[q] = a.out + row_at[pair] * D + half * (D / 2) + 8 * j;
        }
#pragma unroll
        for (int c = 0; c < D / 2; c += 32) {
          uint32_t v[16], w[4];
          if (n > 0) {
            tmem_ld_16x256<4>(o_addr + c + (static_cast<uint32_t>(half16 * 16) << 16), v);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = 0u;
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
              w[g] = pack_bf16x2(__uint_as_float(v[4 * g + 2 * q]) * iv[q], __uint_as_float(v[4 * g + 2 * q + 1]) * iv[q]);
            transpose4(w, j);
            if (mine[q]) *reinterpret_cast<uint4*>(dst[q] + c) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  } else if (FP8) {
    // ---------------------------------------------------------- converters
    const int r = threadIdx.x - 32 * (kRowSoftWarps + 2);
    bool ok = true;
    for (int u = 0; u < 2 * n; ++u) {
      const int s = slot_of(u);
      const uint32_t entry = list[u >> 1];
      const bool zero = (u & 1) && entry >> 24 != 0 && !seen_by_any(offset0(entry) + r);
      if (ok) ok = mbar_wait_inl(full + s, phase_of(u), a.err);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      expand_row(smem + L::kRingOff + s * kSlotBytes, r, D == 128, zero);
      fence_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(ready + s);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

template <bool FP8, int D>
cudaError_t launch_rows(const msa_plan_s* p, ColArgs a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  using L = RowSmem<FP8, D>;
  a.max_groups = (p->max_tile_rows * (p->hq / p->hp) + 255) / 256;
  const int64_t ctas = int64_t(p->n_tiles) * p->hp * a.max_groups;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  auto kern = rows_kernel<FP8, D>;
  static_assert(L::bytes(1024) + 1024 <= 232448, "shared memory at the largest topk");
  static std::atomic<uint64_t> devices{0};
  const uint64_t bit = p->device < 64 ? uint64_t(1) << p->device : 0;
  if ((devices.load(std::memory_order_acquire) & bit) == 0) {
    if (const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes(1024) + 1024))
      return e;
    devices.fetch_or(bit, std::memory_order_release);
  }
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(row_threads<FP8>()), L::bytes(p->topk) + 1024, st, km, vm, a);
}

// Columns a CTA (N), CTAs that share a unit's blocks (parts), and whether two CTAs
// share an SM: the least estimated time over the choices.  A CTA takes about
// start + blocks * step, both measured (us, head_dim 128 or latent_dim 512):
//              start, step        N = 16       32         64        128
//   bf16                         5.6, 0.6   6, 0.68    6.3, 1.05   8.6, 1.72
//   e4m3                         5.2, 0.93  6.4, 1.0   6, 1.65     10.3, 1.87
//   latent                       8.8, 1.95  9.9, 2.08  12.3, 2.41
// (latents of 128, 256 and 384 dims: 0.70, 0.80 and 0.90 of the start, 0.51, 0.68 and 0.84 of the step),
// (1.2 more where bf16 or e4m3 parts merge), and no less than the blocks' bytes take from HBM at 6.3
// TB/s, 3 us of it within the start.  The CTAs run in
// rounds: 152, 76 clusters of 2, 36 of 4, 15 of 8, 7 of 16 at once (large clusters are
// not placed as densely as the SMs would allow).  Two on an SM hide each other's
// start and end where there would be several rounds (bf16 up to 64 columns: 32 x 8
// drafts 54.2 -> 50.1; e4m3, whose converters want the SM, 64.3 -> 67.7; the latent's
// blocks fill the shared memory).  Examples (us, N / parts, all choices tried):
//   16 drafts, 64 / 8 heads, bf16, 16 blocks: 32 / 4 10.3, 64 / 4 11.5, 16 / 2 11.7, 128 / 8 14.2
//   the same, e4m3: 32 / 4 12.0, 64 / 4 14.1, 16 / 2 14.8, 128 / 8 16.2
//   32 x 8 drafts, bf16: 64 / 1 54.2, 128 / 1 65.0, 32 / 1 79.3, 16 / 1 122
//   1 row, 64 heads, latent, 16 blocks: 16 / 16 9.8, 32 / 16 11.8, 16 / 4 15.3, 64 / 8 16.1
//   32 rows, same: 64 / 4 27.2, 32 / 2 29.9, 64 / 2 36.3, 16 / 1 41.4
using Columns = msa_plan_s::Columns;
constexpr double kStreamed = 3;  // us of a start in which blocks stream already
template <int KIND>
Columns column_shape(const msa_plan_s* p, int64_t block_bytes, double size, double& least) {
  static constexpr double kStart[3][4] = {{5.6, 6, 6.3, 8.6}, {5.2, 6.4, 6, 10.3}, {8.8, 9.9, 12.3, 1e9}};
  static constexpr double kStep[3][4] = {{0.6, 0.68, 1.05, 1.72}, {0.93, 1.0, 1.65, 1.87}, {1.95, 2.08, 2.41, 1e9}};
  static constexpr int kClusters[5] = {152, 76, 36, 15, 7};
  const int blocks = std::min(p->max_nvp, p->topk);
  Columns best{16, 1, false, false};
  least = 1e300;
  for (int k = 0; k < (KIND == kLatent ? 3 : 4); ++k) {
    const int64_t units = p->col_units[k], sets = int64_t(p->n_tiles) * p->hp;
    const double start = kStart[KIND][k] * (KIND == kLatent ? 0.55 + 0.45 * size : 1.0);
    auto take = [&](int lg, bool two) {
      const int parts = 1 << lg;
      const int64_t room = std::max<int64_t>(1, int64_t(kClusters[lg]) * (two ? 2 : 1) * p->num_sms / 152);
      const int64_t rounds = (units + room - 1) / room;
      const double at_once = static_cast<double>(std::min(units, room) * parts);
      const double hbm = at_once * block_bytes * sets / units / 6.3e6;  // us a block step
      const double step = kStep[KIND][k] * (KIND == kLatent ? 0.27 + 0.73 * size : size) * (two ? 2.0 : 1.0);
      const int most = (blocks + parts - 1) / parts;
      const double us = rounds * (start + (two ? 2 : 0) + (parts > 1 && KIND != kLatent ? 1.2 : 0) + std::max(most * step, most * hbm - kStreamed));
      if (us < least) best = {16 << k, parts, two, false}, least = us;
    };
    for (int lg = 0; (1 << lg) <= kMaxParts && (1 << lg) <= blocks; ++lg) take(lg, false);
    if (KIND == kBf16 && k < 3) take(0, true);
  }
  return best;
}

// The same estimate for the pairs as rows: 256 a CTA, no parts.  Measured (us; 64 / 8
// heads, 4, 6 and 16 blocks): 128 pairs or fewer a CTA bf16 11.8, 13.7, 29.2, e4m3 12.1,
// 14.6, 29.8, head_dim 64 10.2, 12.0, 24.1; 256 pairs, 152 CTAs, 16 blocks 35, head_dim 64 30.
// As rows, and as columns at their best (bf16; e4m3), 16 blocks:
//    8 x 16 drafts   29.2, 23.1   29.8, 28.1      32 x 8    60.9, 49.5   60.8, 63.3
//    8 x 64          35.6, 65.8   36.1, 82.4      32 x 64   140, -       140, 293
double rows_us(const msa_plan_s* p, int64_t block_bytes, double size) {
  const int64_t units = p->col_units[4], rounds = (units + p->num_sms - 1) / p->num_sms;
  const double at_once = static_cast<double>(std::min<int64_t>(units, p->num_sms));
  const double hbm = at_once * block_bytes * p->n_tiles * p->hp / units / 6.3e6;
  const bool two = p->max_tile_rows * (p->hq / p->hp) > 128;  // tiles a CTA
  const int blocks = std::min(p->max_nvp, p->topk);
  return rounds * ((two ? 8 : 6.1) + std::max(blocks * (two ? 1.7 : 1.47) * size, blocks * hbm - kStreamed));
}

template <int KIND, int N, bool TWO>
cudaError_t launch_columns(const msa_plan_s* p, ColArgs a, const CUtensorMap& km, const CUtensorMap& vm, int parts,
                           cudaStream_t st) {
  using L = ColSmem<KIND, N, TWO>;
  const int groups = (p->max_tile_rows * (p->hq / p->hp) + N - 1) / N;
  a.parts = parts;
  a.max_groups = groups;
  const int64_t ctas = int64_t(p->n_tiles) * p->hp * groups * parts;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  auto kern = columns_kernel<KIND, N, TWO>;
  // Q^T in boxes where the columns of a CTA are whole rows, or lie in one: by 16-byte copies
  // a CTA waits for them behind its first K and V (32 x 8 drafts 51.4 against 50.2 us)
  CUtensorMap qm = km;
  const int G = p->hq / p->hp;
  if (KIND != kE4m3 && (N % G == 0 || G % N == 0)) {
    const uint64_t dims[3] = {static_cast<uint64_t>(a.dq), static_cast<uint64_t>(p->hq), static_cast<uint64_t>(p->total_q)};
    const uint64_t str[2] = {2u * dims[0], 2u * dims[0] * dims[1]};
    const uint32_t box[3] = {64, static_cast<uint32_t>(std::min(G, N)), static_cast<uint32_t>(G < N ? N / G : 1)};
    if (!encode_tensor_map(&qm, 3, a.q, dims, str, box, 1, 128)) return cudaErrorInvalidValue;
    a.q_tma = 1;
  }
  // the limit is the function's, for every host thread: always the most of any topk
  static_assert(L::bytes(1024) + 1024 <= 232448, "shared memory at the largest topk");
  static std::atomic<uint64_t> devices{0};  // that have these limits (the call takes about a microsecond)
  const uint64_t bit = p->device < 64 ? uint64_t(1) << p->device : 0;
  if ((devices.load(std::memory_order_acquire) & bit) == 0) {
    if (const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes(1024) + 1024))
      return e;
    if (const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) return e;
    devices.fetch_or(bit, std::memory_order_release);
  }
  return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(ctas)), parts, dim3(col_threads<KIND, N, TWO>()),
                            L::bytes(p->topk) + 1024, st, km, vm, qm, a);
}

template <int KIND>
cudaError_t launch_shape(Columns c, const msa_plan_s* p, const ColArgs& a, const CUtensorMap& km, const CUtensorMap& vm,
                         cudaStream_t st) {
  if constexpr (KIND == kBf16)
    if (c.two)
      return c.n == 16   ? launch_columns<KIND, 16, true>(p, a, km, vm, 1, st)
             : c.n == 32 ? launch_columns<KIND, 32, true>(p, a, km, vm, 1, st)
                         : launch_columns<KIND, 64, true>(p, a, km, vm, 1, st);
  if constexpr (KIND != kLatent)
    if (c.n == 128) return launch_columns<KIND, 128, false>(p, a, km, vm, c.parts, st);
  return c.n == 16   ? launch_columns<KIND, 16, false>(p, a, km, vm, c.parts, st)
         : c.n == 32 ? launch_columns<KIND, 32, false>(p, a, km, vm, c.parts, st)
                     : launch_columns<KIND, 64, false>(p, a, km, vm, c.parts, st);
}

}  // namespace

void column_plan_counts(msa_plan_s* p) {
  const int G = p->hq / p->hp;
  for (const TileInfo& t : p->tiles) {
    p->max_tile_rows = std::max(p->max_tile_rows, t.rows);
    p->max_nvp = std::max(p->max_nvp, t.nvp);
    for (int k = 0; k < 5; ++k) p->col_units[k] += int64_t(p->hp) * ((int64_t(t.rows) * G + (16 << k) - 1) >> (4 + k));
  }
  const bool fp8 = p->kv_dtype != MSA_KV_BF16;
  const int64_t bytes = int64_t(256) * p->d * (fp8 ? 1 : 2);
  const double size = p->d == 128 ? 1.0 : 0.87;
  double us;
  p->tree_shape = fp8 ? column_shape<kE4m3>(p, bytes, size, us) : column_shape<kBf16>(p, bytes, size, us);
  p->tree_shape.rows = rows_us(p, bytes, size) < us;
  for (int k = 0; k < 4; ++k) {  // (with the widest rotated part: blocks of 128 dims are a quarter smaller at most, of 512 8 %)
    const int width = 128 * (k + 1) + 64;
    p->latent_shape[k] = column_shape<kLatent>(p, int64_t(256) * width, width / 576.0, us);
  }
}

msa_status launch_tree_attn(const msa_plan_s* p, const void* q, const void* k_pages, const void* v_pages,
                            const int32_t* kv_indices, const int32_t* idx, const int32_t* tree_mask, const float* k_scale,
                            const float* v_scale, void* out, float* lse, cudaStream_t st) {
  const bool fp8 = p->kv_dtype != MSA_KV_BF16;
  CUtensorMap km, vm;
  // bf16: a block in one load, 64 columns (128-byte rows) after the other; e4m3: whole rows of codes
  const uint64_t rows = static_cast<uint64_t>(p->num_pages) * p->hkv * 128, d = p->d;
  const uint64_t dims[3] = {fp8 ? d : 64, rows, d / 64};
  const uint64_t str[2] = {d * (fp8 ? 1 : 2), 128};
  const uint32_t box[3] = {static_cast<uint32_t>(dims[0]), 128, static_cast<uint32_t>(d / 64)};
  const int swz = fp8 ? p->d : 128, rank = fp8 ? 2 : 3;
  if (!encode_tensor_map(&km, rank, k_pages, dims, str, box, fp8 ? 0 : 1, swz) ||
      !encode_tensor_map(&vm, rank, v_pages, dims, str, box, fp8 ? 0 : 1, swz))
    return set_error(MSA_ERR_CUDA, "msa_tree_attn: tensor map encoding failed");
  ColArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.tiles = p->tiles_d;
  a.idx = idx;
  a.kv_indices = kv_indices;
  a.tree_mask = reinterpret_cast<const uint32_t*>(tree_mask);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.err = p->err_d;
  a.num_pages = p->num_pages;
  a.hq = p->hq, a.hp = p->hp, a.hkv = p->hkv;
  a.topk = p->topk;
  a.dq = a.dv = p->d;
  a.kc = p->d / 64;
  a.mt = 1;
  a.per_page = p->kv_dtype == MSA_KV_FP8_E4M3_BLOCK;
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(p->d));
  const Columns& shape = p->tree_shape;
  const cudaError_t e = shape.rows ? (fp8 ? (p->d == 128 ? launch_rows<true, 128>(p, a, km, vm, st) : launch_rows<true, 64>(p, a, km, vm, st))
                                          : (p->d == 128 ? launch_rows<false, 128>(p, a, km, vm, st) : launch_rows<false, 64>(p, a, km, vm, st)))
                        : fp8      ? launch_shape<kE4m3>(shape, p, a, km, vm, st)
                                   : launch_shape<kBf16>(shape, p, a, km, vm, st);
  return cuda_check(e, "msa_tree_attn: launch");
}

msa_status launch_latent_attn(const msa_plan_s* p, const void* q, const void* latent_pages, const int32_t* kv_indices,
                              const int32_t* idx, const int32_t* tree_mask, int32_t latent_dim, int32_t rope_dim,
                              float scale, void* out, float* lse, cudaStream_t st) {
  CUtensorMap km, vm;
  const int width = latent_dim + rope_dim;
  // the rotated part: a box of 64 columns, those past the row zeros; the latent's
  // 128 dims of a slot: two boxes of 64 columns in one load
  const uint64_t rows = static_cast<uint64_t>(p->num_pages) * 128;
  const uint64_t dims[2] = {static_cast<uint64_t>(width), rows}, dims3[3] = {64, rows, static_cast<uint64_t>(latent_dim / 64)};
  const uint64_t str[2] = {static_cast<uint64_t>(width) * 2, 128};
  const uint32_t box[2] = {64, 128}, box3[3] = {64, 128, 2};
  if (!encode_tensor_map(&km, 2, latent_pages, dims, str, box, 1, 128) ||
      !encode_tensor_map(&vm, 3, latent_pages, dims3, str, box3, 1, 128))
    return set_error(MSA_ERR_CUDA, "msa_latent_attn: tensor map encoding failed");
  ColArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.tiles = p->tiles_d;
  a.idx = idx;
  a.kv_indices = kv_indices;
  a.tree_mask = reinterpret_cast<const uint32_t*>(tree_mask);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.err = p->err_d;
  a.num_pages = p->num_pages;
  a.hq = p->hq, a.hp = p->hp, a.hkv = 1;
  a.topk = p->topk;
  a.dq = width;
  a.dv = latent_dim;
  a.kc = latent_dim / 64 + 1;
  a.mt = latent_dim / 128;
  a.scale_log2 = 1.4426950408889634f * scale;
  return cuda_check(launch_shape<kLatent>(p->latent_shape[latent_dim / 128 - 1], p, a, km, vm, st), "msa_latent_attn: launch");
}

namespace {

// The tiles of a tree are its sequence's drafts: one tile a sequence, whose
// masks have 128 bits.
msa_status check_tree(const char* fn, const msa_plan_s* p) {
  for (int32_t n : p->qo_lens)
    if (n > kTile) return set_error(MSA_ERR_UNSUPPORTED, "%s: a tree has at most %d drafts, a sequence has %d", fn, kTile, n);
  return MSA_OK;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

}  // namespace msa

using namespace msa;

extern "C" {

msa_status msa_tree_attn(msa_plan_t plan, const void* q, const void* k_pages, const void* v_pages,
                         const int32_t* kv_indices, const int32_t* kv_block_indexes, const int32_t* tree_mask,
                         const float* k_scale, const float* v_scale, void* out, float* lse, msa_stream_t stream) {
  const char* fn = "msa_tree_attn";
  if (!plan || !q || !k_pages || !v_pages || !kv_indices || !kv_block_indexes || !tree_mask || !out)
    return set_error(MSA_ERR_INVALID_ARG, "%s: NULL argument", fn);
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
    return set_error(MSA_ERR_INVALID_ARG, "%s: q, k_pages, v_pages, out must be 16-byte aligned", fn);
  if (!aligned4(tree_mask)) return set_error(MSA_ERR_INVALID_ARG, "%s: tree_mask must be 4-byte aligned", fn);
  const bool fp8 = plan->kv_dtype != MSA_KV_BF16;
  if (fp8 != (k_scale != nullptr) || fp8 != (v_scale != nullptr))
    return set_error(MSA_ERR_INVALID_ARG, "%s: k_scale/v_scale must be given exactly for FP8 K/V", fn);
  // K/V rows are 32-bit coordinates of the loads, which read zeros beyond them.  (A latent
  // cache has one head, and a plan at most 2^24 pages.)
  if (plan->num_pages * plan->hkv > (int64_t(1) << 24))
    return set_error(MSA_ERR_INVALID_ARG, "%s: num_pages * num_kv_heads above 2^24", fn);
  msa_status s = check_tree(fn, plan);
  if (s == MSA_OK) s = check_device(fn, plan);
  if (s != MSA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  s = launch_tree_attn(plan, q, k_pages, v_pages, kv_indices, kv_block_indexes, tree_mask, k_scale, v_scale, out, lse, st);
  const int64_t rows = plan->total_q * plan->hq;
  if (s == MSA_OK) s = scan_rows(plan, q, rows * plan->d, 2, st);
  if (s == MSA_OK) s = scan_rows(plan, out, rows * plan->d, 2, st);
  if (s == MSA_OK) s = scan_rows(plan, lse, rows, 4, st);
  return s;
}

msa_status msa_latent_attn(msa_plan_t plan, const void* q, const void* latent_pages, const int32_t* kv_indices,
                           const int32_t* kv_block_indexes, const int32_t* tree_mask, int32_t latent_dim,
                           int32_t rope_dim, float scale, void* out, float* lse, msa_stream_t stream) {
  const char* fn = "msa_latent_attn";
  if (!plan || !q || !latent_pages || !kv_indices || !kv_block_indexes || !out)
    return set_error(MSA_ERR_INVALID_ARG, "%s: NULL argument", fn);
  if (const msa_status s = check_latent_dims(fn, latent_dim, rope_dim); s != MSA_OK) return s;
  if (!(scale > 0.f) || !(scale < INFINITY)) return set_error(MSA_ERR_INVALID_ARG, "%s: scale must be positive", fn);
  if (!aligned16(q) || !aligned16(latent_pages) || !aligned16(out))
    return set_error(MSA_ERR_INVALID_ARG, "%s: q, latent_pages, out must be 16-byte aligned", fn);
  if (!aligned4(tree_mask)) return set_error(MSA_ERR_INVALID_ARG, "%s: tree_mask must be 4-byte aligned", fn);
  msa_status s = tree_mask ? check_tree(fn, plan) : MSA_OK;
  if (s == MSA_OK) s = check_device(fn, plan);
  if (s != MSA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  s = launch_latent_attn(plan, q, latent_pages, kv_indices, kv_block_indexes, tree_mask, latent_dim, rope_dim, scale, out,
                         lse, st);
  const int64_t rows = plan->total_q * plan->hq;
  if (s == MSA_OK) s = scan_rows(plan, q, rows * (latent_dim + rope_dim), 2, st);
  if (s == MSA_OK) s = scan_rows(plan, out, rows * latent_dim, 2, st);
  if (s == MSA_OK) s = scan_rows(plan, lse, rows, 4, st);
  return s;
}

}  // extern "C"
