// Stage 3 (prefill): GQA block-sparse flash attention forward, bf16 or FP8 K/V.
//
// For query row i of tile t and head h (KV head g = h / (Hq/Hkv), proxy
// head p = h / (Hq/Hp)): softmax over the keys of the selected blocks
// kv_block_indexes[t, p, :] that are visible to i, of q.k_g/sqrt(d); out =
// P.V_g and lse = ln sum exp ("MiniMax-AI/MSA" README, section "Usage":
// fmha_sm100(q, k_pages, v_pages, sparse_plan, kv_indices,
// kv_block_indexes); Flash-MSA article, "three key differences": the main
// attention is GQA and each proxy head picks its own block set).  With one
// proxy head per GQA group, p = g.
//
// A work unit is (tile, proxy head, pair of the query heads that use its
// blocks): both heads share every K/V block the TMA producer gathers
// through the page table.  Tensor memory holds S0, S1 (128 columns each) and O0, O1 (d
// columns each); the bf16 probabilities P_h overwrite the first 64 columns
// of S_h and feed the P.V MMA straight from tensor memory.  Roles:
//   warps 0-3  softmax of head 0 (thread = query row), warps 4-7 head 1,
//   warp 8     producer: builds each unit's block list (top-k row and page
//              rows, all 32 lanes at once) into a two-slot ring, loads Q per
//              unit and the K/V blocks into a 2-stage ring (one barrier per
//              stage for K and V),
//   warp 9     MMA issuer: S_h = Q_h K^T (smem x smem), O_h += P_h V
//              (tmem x smem), ordered QK0 QK1 | PV0 QK0' PV1 QK1' | ... so
//              that one head's softmax overlaps the other head's MMAs.
// The issuing thread runs only about one MMA ahead of the tensor pipe, so
// its loop does nothing between MMA groups that it can avoid: three waits
// and three commits per block step, descriptors precomputed.
// Online softmax in the log2 domain; the O rescale runs in the softmax
// warps between P.V steps, and the epilogue releases O_h to the next unit
// as soon as it is in registers.
//
// FP8 K/V ("MiniMax-AI/MSA" README, section "Stacks": sparse prefill in FP8
// next to BF16).  K/V pages hold e4m3 codes with one fp32 scale per KV
// head: logit = (q . k_code) * k_scale / sqrt(d), v = v_code * v_scale.  The
// producer gathers the 16 KB code blocks by TMA into the upper half of the
// K / V ring stages, and two converter warps (warps 10-11) expand them in
// place to f16 (exact: every e4m3 value is an f16) in the 128-byte-swizzled
// layout the MMAs read, and convert each unit's Q tiles in place from bf16
// to f16.  The MMAs then run kind::f16 with f16 operands (Q, K, P and V),
// k_scale folds into the softmax scale and v_scale into the epilogue.
// Rounding: Q to f16 is exact for |q| in [2^-14, 65504] (smaller values
// lose at most 2^-25, larger ones saturate) and P is rounded to f16 instead
// of bf16.
//
// kBlk: one scale for each (page, KV head) instead (BlockScale in
// msa_internal.h).  The producer's lanes fetch them beside the page ids, at
// least 32 blocks ahead, into a ring that the softmax warps read, one pair a
// block, into the multiply-add that scales the logits (fetched and converted
// by the softmax warps themselves they cost 130 us of 965 at S=32768).  The
// converters write zeros for V rows behind the sequence's last key, whose
// bytes were never written.
//
// kSplit (kBlk, few units): the CTAs of a cluster take a part of one unit's
// blocks each, leave their O, m and l in shared memory (where the rings were)
// and merge a share of the rows each over distributed shared memory.
#include "msa_internal.h"
#include "ptx.cuh"

#include <algorithm>

namespace msa {
namespace {

constexpr int kStages = 2;
constexpr int kSoftWarps = 8;
constexpr int kConvWarps = 2;  // FP8 K/V only
constexpr int kEpiWarp0 = 12;  // warps 12-15: epilogue
constexpr int kMaxTopk = 1024;
// Four warpgroups: softmax (two), producer / MMA / FP8 converters, epilogue.
// Launched at 128 registers a thread; the softmax warpgroups then take
// kSoftRegs and the other two give theirs back down to kWg2Regs and
// kEpiRegs, which adds up to the launch's 512 x 128 (an increase waits for
// the decreases otherwise).
constexpr int kAttnThreads = 512;
constexpr int kLaunchRegs = 128;
constexpr int kSoftRegs = 168;
constexpr int kWg2Regs = 104;
constexpr int kEpiRegs = 72;
static_assert(256 * kSoftRegs + 128 * kWg2Regs + 128 * kEpiRegs == kAttnThreads * kLaunchRegs, "register split");

struct AttnUnit {
  int32_t tile, g, h0;
  int16_t nh, lg;
};
static_assert(sizeof(AttnUnit) == 16, "four words of the plan's aux array");

// The queries' tensor maps: [lg] has boxes of 2^lg heads x 128 >> lg rows.
constexpr int kMaxPack = 4;
template <bool kBlk>
struct QueryMaps {
  CUtensorMap by_lg[kBlk ? kMaxPack + 1 : 1];
};

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  tmem_st16(taddr, r);
  tmem_st16(taddr + 16, r + 16);
}

// One unit's cached blocks, built once by the producer warp (its lanes read
// the top-k row and the page table in parallel) for the MMA and softmax
// warps: a 16-int header, then j[cap] (selected blocks, padding and
// out-of-range entries dropped) and row[cap] (their first K/V tensor-map
// row), cap >= topk.
struct UnitHdr {
  int32_t n, nh, h0, q_begin, rows, pos0, g, kv_len, h_end, lg, pad[6];
};
constexpr int kListSlots = 2;
constexpr int kScaleRing = 128;  // blocks; written up to 64 ahead of the one being loaded
constexpr int kHdrInts = 16;

// A head's row statistics at the end of a unit, from the softmax warps to
// the epilogue warps (two buffers per head, alternating by unit).
struct UnitStats {
  int32_t n, active, ok, h0, q_begin, rows, g, h_end, lg, pad[7];
  float m[128], l[128];
};

// Shared memory: Q (two heads), the K and V rings, the O staging buffer
// (kStageO: one 64-column box of a head's bf16 O tile, for the TMA stores of
// full tiles), barriers, the units' row statistics, then the two list slots,
// whose size follows topk.
template <int D, bool kStageO, int kLists = 1, bool kBlk = false>
struct AttnSmem {
  static constexpr int kTileBytes = 128 * D * 2;  // 128 rows x D bf16, in D/64 swizzled chunks of 16 KB
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kStages * kTileBytes;
  static constexpr int kOOff = kVOff + kStages * kTileBytes;
  static constexpr int kOChunkBytes = 128 * 64 * 2;  // 64 columns of 128 rows
  static constexpr int kBarOff = kOOff + (kStageO ? kOChunkBytes : 0);
  static constexpr int kStatOff = kBarOff + 8 * 64;
  static constexpr int kScaleOff = kStatOff + 4 * static_cast<int>(sizeof(UnitStats));
  static constexpr int kListOff = kScaleOff + (kBlk ? 8 * kScaleRing : 0);
  static __host__ __device__ constexpr int slot_ints(int cap) { return kHdrInts + 2 * kLists * cap; }
  static __host__ __device__ constexpr int bytes(int cap) { return kListOff + kListSlots * slot_ints(cap) * 4; }
};

// Persistent: CTA b takes units b, b + gridDim.x, ... (heaviest first).
// Tensor memory, barriers and the K/V ring live across units; every
// barrier's phase comes from a running count (per head for the S / P / O
// barriers), and Q is released right after a unit's last QK so the next
// unit's Q load overlaps the tail of the current one.
template <int D, bool kOneKvHead, bool kFp8, bool kStageO, bool kBlk = false, bool kSplit = false, bool kLead = false>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_fwd_kernel(const __grid_constant__ QueryMaps<kBlk> q_maps, const __grid_constant__ CUtensorMap k_map,
                    const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap o_map,
                    int32_t list_cap, const AttnUnit* __restrict__ units, int32_t n_units,
                    const TileInfo* __restrict__ tiles, const int32_t* __restrict__ idx,
                    const int32_t* __restrict__ kv_indices, int64_t num_pages, __nv_bfloat16* __restrict__ out,
                    float* __restrict__ lse, int32_t hq, int32_t hsel, int32_t kv_div, int32_t topk,
                    float scale_log2, const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                    int32_t parts, uint32_t* err, int32_t chain) {
  if (kSplit && (chain & kFollows))
    fence_gpu();
  else
    pdl_wait();
  // a variant of its own: the call alone costs the others 1 % (32K prefill 862 -> 870 us)
  if (kLead || (kSplit && (chain & kLeads))) pdl_trigger();
  // kBlk: a unit of a tile of few rows has 2^lg heads side by side in the 128
  // rows of a product, row r being query row r >> lg of head r % 2^lg; "head" 0
  // and 1 of a unit are then such groups
  // kSplit (few units): a unit's blocks are shared out over the `parts` CTAs of
  // a cluster, which do nothing else and merge at the end
  const int part = kSplit ? blockIdx.x % parts : 0;
  auto first_unit = [&]() -> int { return kSplit ? blockIdx.x / parts : blockIdx.x; };
  // hsel block sets (proxy heads) per tile; a unit's u.g is its proxy head,
  // whose blocks are read from KV head u.g / kv_div of hsel / kv_div
  const int hkv = hsel / kv_div;
  // a one-head K/V pool (the backward's proxy softmax) pairs two proxy heads
  // per unit, each over its own blocks: one (j, row) list per head
  using L = AttnSmem<D, kStageO, kOneKvHead ? 2 : 1, kBlk>;
  constexpr int kChunks = D / 64;
  static_assert(!kFp8 || ((D == 128 || kBlk) && !kOneKvHead), "FP8 K/V: head_dim 128 or block scales, main attention");
  static_assert(!kBlk || kFp8, "block scales come with FP8 K/V");
  static_assert(!kSplit || (kBlk && !kStageO), "split units: block scales, O through the merge");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem + L::kQOff;
  uint8_t* k_s = smem + L::kKOff;
  uint8_t* v_s = smem + L::kVOff;
  int32_t* const list_base = reinterpret_cast<int32_t*>(smem + L::kListOff);
  // A part's O_h: rows of D floats where the K (h = 0) or V ring was, their
  // 16-byte chunks spread over the banks by row.  P_0.V of the unit's last
  // block is issued after its last Q K^T, and P_1.V after that: the K ring is
  // free once O_0 is done, the V ring once O_1 is.
  auto part_o = [](uint8_t* base, int h, int r, int chunk) -> uint4& {
    return reinterpret_cast<uint4*>(base + (h == 0 ? L::kKOff : L::kVOff))[r * (D / 4) + (chunk ^ (r & (D / 4 - 1)))];
  };
  // the staged layout sizes the list slots by topk; the other keeps them at
  // the compile-time maximum (constant offsets in the issue loops)
  const int cap = kStageO ? list_cap : kMaxTopk;
  const int slot_ints = L::slot_ints(cap);
  auto lhdr = [&](int k) -> UnitHdr& { return *reinterpret_cast<UnitHdr*>(list_base + (k % kListSlots) * slot_ints); };
  auto lj = [&](int k) -> int32_t* { return list_base + (k % kListSlots) * slot_ints + kHdrInts; };
  auto lrow = [&](int k) -> int32_t* { return list_base + (k % kListSlots) * slot_ints + kHdrInts + cap; };
  auto lj1 = [&](int k) -> int32_t* { return list_base + (k % kListSlots) * slot_ints + kHdrInts + 2 * cap; };
  auto lrow1 = [&](int k) -> int32_t* { return list_base + (k % kListSlots) * slot_ints + kHdrInts + 3 * cap; };
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* kv_full = bars + 2;              // [kStages]: K and V of a block
  uint64_t* kv_empty = kv_full + kStages;
  uint64_t* s_full = kv_empty + kStages;  // [2]
  uint64_t* p_full = s_full + 2;          // [2]
  uint64_t* o_done = p_full + 2;          // [2]: a unit's last P.V of head h
  uint64_t* o_free = o_done + 2;          // [2]: the epilogue has read a unit's O_h (units with blocks, either head)
  uint64_t* list_full = o_free + 2;       // [kListSlots]
  uint64_t* list_empty = list_full + kListSlots;
  uint64_t* drain = list_empty + kListSlots;
  uint64_t* raw_full = drain + 1;          // [kStages], FP8: e4m3 K and V codes landed
  uint64_t* q_ready = raw_full + kStages;  // FP8: Q converted to f16
  uint64_t* ost_ready = q_ready + 1;       // a head's O staged (kStageO)
  uint64_t* ost_free = ost_ready + 1;      // the TMA store has read it
  uint64_t* stat_full = ost_free + 1;      // [head * 2 + buffer]
  uint64_t* stat_empty = stat_full + 4;    // [head * 2 + buffer]
  // FP8: K and V of a block travel apart, kv_full / kv_empty / raw_full being
  // one half's (a block's K is read for the last time by S_1 = Q_1 K^T, a whole
  // step before P_1 V reads its V, and each half has to be loaded and then
  // expanded within the time from its release to its next use)
  uint64_t* k_full = kv_full;              // [kStages]
  uint64_t* k_empty = stat_empty + 4;      // [kStages]
  uint64_t* v_full = k_empty + kStages;    // [kStages]
  uint64_t* v_empty = kv_empty;            // [kStages]
  uint64_t* raw_v_full = v_full + kStages; // [kStages]
  uint64_t* conv_read = raw_v_full + kStages;  // head_dim 64: both converter warps hold a half's codes
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(conv_read + 1);
  UnitStats* const stats = reinterpret_cast<UnitStats*>(smem + L::kStatOff);
  // kBlk: (k_scale * scale_log2, log2 v_scale) of the running block count's block
  float2* const scale_ring = reinterpret_cast<float2*>(smem + L::kScaleOff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    if (!kBlk) prefetch_tmap(&q_maps.by_lg[0]);  // kBlk: the producer, which knows the unit's
    prefetch_tmap(&k_map);
    prefetch_tmap(&v_map);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(kv_full + s, kFp8 ? kConvWarps : 1);
      mbar_init(kv_empty + s, 1);
      mbar_init(raw_full + s, 1);
      mbar_init(k_empty + s, 1);
      mbar_init(v_full + s, kConvWarps);
      mbar_init(raw_v_full + s, 1);
    }
    mbar_init(q_ready, kConvWarps);
    mbar_init(conv_read, kConvWarps);
    mbar_init(ost_ready, 4);  // the four epilogue warps
    mbar_init(ost_free, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(stat_full + i, 4);   // the head's four softmax warps
      mbar_init(stat_empty + i, 4);  // the four epilogue warps
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(s_full + h, 1);
      mbar_init(p_full + h, 4);
      mbar_init(o_done + h, 1);
      mbar_init(o_free + h, 4);  // the epilogue warps
    }
    for (int i = 0; i < kListSlots; ++i) {
      mbar_init(list_full + i, 1);
      mbar_init(list_empty + i, 1 + kSoftWarps + (kFp8 ? kConvWarps : 0));  // MMA thread, softmax (and converter) warps
    }
    mbar_init(drain, 1);
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
  // each role's branch starts with its warpgroup's register share

  if (warp == 8) {
    // ---------------------------------------------------------- producer
    setmaxnreg_dec<kWg2Regs>();
    int kv_it = 0;
    bool ok = true;
    auto put_scale = [&](int it, int row) {
      const BlockScale b = block_scale_of(k_scale[row >> 7], v_scale[row >> 7]);
      scale_ring[it % kScaleRing] = make_float2(b.ks * scale_log2, b.log2_vs);
    };
    for (int k = 0, ui = first_unit(); ok && ui < n_units; ++k, ui += kSplit ? n_units : gridDim.x) {
      UnitHdr& ls = lhdr(k);
      int32_t* const ls_j = lj(k);
      int32_t* const ls_row = lrow(k);
      const AttnUnit u = units[ui];
      const TileInfo tl = tiles[u.tile];
      const int lg = kBlk ? u.lg : 0;
      if (kBlk && k == 0 && lane == 0) prefetch_tmap(&q_maps.by_lg[lg]);
      const int32_t* sel = idx + (static_cast<int64_t>(u.tile) * hsel + u.g) * topk;
      if (lane == 0) ok = mbar_wait_inl(list_empty + k % kListSlots, ((k / kListSlots) & 1) ^ 1, err);
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      __syncwarp();
      if (!ok) break;
      // the unit's blocks: padding skipped, entries past the tile's valid
      // blocks dropped and reported, pages checked against the pool (kBlk: a
      // block on a page outside is dropped; otherwise page 0 is read in its place)
      int first = 0, count = topk, seen = 0;  // of the valid blocks, this part's
      if (kSplit) {
        int total = 0;
        for (int b = 0; b < topk; b += 32) {
          const int j = b + lane < topk ? sel[b + lane] : -1;
          total += __popc(__ballot_sync(0xFFFFFFFFu, j >= 0 && j < tl.nvp));
        }
        first = total * part / parts;
        count = total * (part + 1) / parts - first;
      }
      int n = 0;
      for (int b = 0; b < topk; b += 32) {
        const int kk = b + lane;
        const int j = kk < topk ? sel[kk] : -1;
        const bool valid = j >= 0 && j < tl.nvp;
        if (j >= tl.nvp) atomicOr(err, kErrDeviceCheck);
        bool take = valid;
        int row = 0;
        if (valid) {
          int64_t page = kv_indices[tl.page_base + j];
          if (page < 0 || page >= num_pages) {
            atomicOr(err, kErrDeviceCheck);
            page = 0;
            if (kBlk) take = false;
          }
          // K/V head of the unit's proxy head, or the single head of a one-head pool
          row = static_cast<int>((kOneKvHead ? page : page * hkv + u.g / kv_div) * 128);
        }
        const uint32_t below = (1u << lane) - 1u;
        if (kSplit) {
          const uint32_t v = __ballot_sync(0xFFFFFFFFu, valid);
          const int rank = seen + __popc(v & below);
          take = take && rank >= first && rank < first + count;
          seen += __popc(v);
        }
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, take);
        if (take) {
          const int o = n + __popc(m & below);
          ls_j[o] = j;
          ls_row[o] = row;
          if (kBlk && o < 64) put_scale(kv_it + o, row);
        }
        n += __popc(m);
      }
      const bool pair = kOneKvHead && u.nh == 2;
      if (pair) {
        // the second proxy head's own blocks (selection row g + 1); the
        // shorter list is padded with j = -1 (fully masked, page row 0)
        int32_t* const ls_j1 = lj1(k);
        int32_t* const ls_row1 = lrow1(k);
        const int32_t* sel1 = sel + topk;
        int n1 = 0;
        for (int b = 0; b < topk; b += 32) {
          const int kk = b + lane;
          const int j = kk < topk ? sel1[kk] : -1;
          const bool valid = j >= 0 && j < tl.nvp;
          if (j >= tl.nvp) atomicOr(err, kErrDeviceCheck);
          int row = 0;
          if (valid) {
            int64_t page = kv_indices[tl.page_base + j];
            if (page < 0 || page >= num_pages) {
              atomicOr(err, kErrDeviceCheck);
              page = 0;
            }
            row = static_cast<int>(page * 128);
          }
          const uint32_t m = __ballot_sync(0xFFFFFFFFu, valid);
          if (valid) {
            const int o = n1 + __popc(m & ((1u << lane) - 1u));
            ls_j1[o] = j;
            ls_row1[o] = row;
          }
          n1 += __popc(m);
        }
        for (int i = n + lane; i < n1; i += 32) {
          ls_j[i] = -1;
          ls_row[i] = 0;
        }
        for (int i = n1 + lane; i < n; i += 32) {
          ls_j1[i] = -1;
          ls_row1[i] = 0;
        }
        n = n > n1 ? n : n1;
      }
      if (lane == 0) {
        ls.n = n;
        ls.nh = u.nh;
        ls.h0 = u.h0;
        ls.q_begin = tl.q_begin;
        ls.rows = tl.rows;
        ls.pos0 = tl.pos0;
        ls.g = u.g / kv_div;
        ls.kv_len = tl.kv_len;
        ls.h_end = (u.g + 1) * (hq / hsel);
        ls.lg = lg;
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(list_full + k % kListSlots);
        if (k > 0) ok = mbar_wait_inl(q_empty, (k - 1) & 1, err);
        if (ok) {
          mbar_expect_tx(q_full, u.nh * L::kTileBytes);
          for (int h = 0; h < u.nh; ++h)
            for (int c = 0; c < kChunks; ++c)
              tma_load_3d(q_s + h * L::kTileBytes + c * 16384, &q_maps.by_lg[lg], q_full, c * 64, u.h0 + (h << lg),
                          tl.q_begin);
        }
      }
      constexpr int kStep = kBlk ? 32 : 1 << 30;  // kBlk: the lanes come together every 32 blocks to fetch scales
      for (int i0 = 0; i0 < n; i0 += kStep) {
        if (kBlk && i0 > 0) {
          if (i0 + 32 + lane < n) put_scale(kv_it + 32 + lane, ls_row[i0 + 32 + lane]);
          ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
          __syncwarp();
        }
        const int i1 = kBlk ? min(n, i0 + kStep) : n;
        for (int i = i0; lane == 0 && ok && i < i1; ++i, ++kv_it) {
          const int s = kv_it % kStages;
          const int row = ls_row[i];
          if (kFp8) {  // e4m3 codes into the upper half of the stage; the converters expand them
            const uint32_t par = ((kv_it / kStages) & 1) ^ 1;
            if (!(ok = mbar_wait_inl(k_empty + s, par, err))) break;
            mbar_expect_tx(raw_full + s, L::kTileBytes / 2);
            tma_load_2d(k_s + s * L::kTileBytes + L::kTileBytes / 2, &k_map, raw_full + s, 0, row);
            if (!(ok = mbar_wait_inl(v_empty + s, par, err))) break;
            mbar_expect_tx(raw_v_full + s, L::kTileBytes / 2);
            tma_load_2d(v_s + s * L::kTileBytes + L::kTileBytes / 2, &v_map, raw_v_full + s, 0, row);
            continue;
          }
          if (!(ok = mbar_wait_inl(kv_empty + s, ((kv_it / kStages) & 1) ^ 1, err))) break;
          // a one-head pool's keys are its values: one load serves both, and
          // a paired unit's second head reads its own block from the V region
          const bool pair = kOneKvHead && u.nh == 2;
          const int row1 = pair ? lrow1(k)[i] : row;
          mbar_expect_tx(kv_full + s, (kOneKvHead && !pair ? 1 : 2) * L::kTileBytes);
          for (int c = 0; c < kChunks; ++c)
            tma_load_2d(k_s + s * L::kTileBytes + c * 16384, &k_map, kv_full + s, c * 64, row);
          if (!kOneKvHead || pair)
            for (int c = 0; c < kChunks; ++c)
              tma_load_2d(v_s + s * L::kTileBytes + c * 16384, &v_map, kv_full + s, c * 64, row1);
        }
        if (kBlk && lane != 0) kv_it += i1 - i0;
        if (!kBlk) break;
      }
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
    }
  } else if (warp == 9) {
    // --------------------------------------------------------------- MMA
    setmaxnreg_dec<kWg2Regs>();
    if (lane == 0) {
      // The issuing thread runs only a step ahead of the tensor pipe, so
      // anything between two MMA groups (a wait, a commit, address
      // arithmetic) idles the pipe: descriptors are precomputed, K and V of
      // a block share one barrier, O_h's barrier is committed once per unit
      // (a block's S_h commit already covers the previous P_h.V), and the
      // per-head phase counters are scalars.
      constexpr uint32_t id_qk = kFp8 ? idesc_f16_f32(128, 128, false, false) : idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t id_pv = kFp8 ? idesc_f16_f32(128, D, false, true) : idesc_bf16_f32(128, D, false, true);
      constexpr uint64_t kTileDesc = L::kTileBytes >> 4;
      const uint64_t qd0 = smem_desc(smem_u32(q_s), 16, 1024, kSwizzle128);
      const uint64_t kd0 = smem_desc(smem_u32(k_s), 16, 1024, kSwizzle128);
      const uint64_t vd0 = smem_desc(smem_u32(kOneKvHead ? k_s : v_s), 16384, 1024, kSwizzle128);
      // a paired one-head unit: head 1's block sits in the V region, as its
      // keys (K-major) and its values (rows-major)
      const uint64_t kd1 = smem_desc(smem_u32(v_s), 16, 1024, kSwizzle128);
      const uint64_t vd1 = smem_desc(smem_u32(v_s), 16384, 1024, kSwizzle128);
      auto qk = [&](int h, int s) {
        const uint64_t qd = qd0 + h * kTileDesc, kd = (kOneKvHead && h == 1 ? kd1 : kd0) + s * kTileDesc;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
          mma_ss(tmem + h * 128, qd + off, kd + off, id_qk, kk > 0);
        }
        mma_commit(s_full + h);
      };
      auto pv = [&](int h, int s, bool acc) {
        const uint64_t vd = (kOneKvHead && h == 1 ? vd1 : vd0) + s * kTileDesc;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + 256 + h * D, tmem + h * 128 + kk * 8, vd + ((kk * 2048) >> 4), id_pv, acc || (kk > 0));
      };
      int kv_it = 0, ch0 = 0, ch1 = 0, used = 0;  // used: units with blocks so far
      bool ok = true;
      for (int k = 0, ui = first_unit(); ok && ui < n_units; ++k, ui += kSplit ? n_units : gridDim.x) {
        if (!(ok = mbar_wait_inl(list_full + k % kListSlots, (k / kListSlots) & 1, err))) break;
        const int n = lhdr(k).n;
        const bool two = lhdr(k).nh == 2;
        mbar_arrive(list_empty + k % kListSlots);
        if (!(ok = mbar_wait_inl(kFp8 ? q_ready : q_full, k & 1, err))) break;
        tc_fence_after();
        // A unit without blocks takes no part in o_done and o_free: what the
        // epilogue does for it waits for nothing of this thread's, so a release of
        // its own could complete before the wait for the one before it, and a
        // parity wait two phases behind waits for ever or ends early.  Every
        // other unit's release follows its o_done, committed after that wait.
        if (n == 0) {
          mma_commit(q_empty);
          continue;
        }
        if (!(ok = mbar_wait_inl(kv_full + (kv_it & 1), (kv_it >> 1) & 1, err))) break;
        tc_fence_after();
        qk(0, kv_it & 1);
        if (two) qk(1, kv_it & 1);
        if (kFp8) mma_commit(k_empty + (kv_it & 1));
        if (n == 1) mma_commit(q_empty);  // the unit's last QK is issued
        for (int i = 0; i < n; ++i) {
          const int it = kv_it + i;
          const int s = it & 1, s1 = s ^ 1;
          const bool more = i + 1 < n;
          // head 0: P_0 . V, then S_0 of the next block
          if (!(ok = mbar_wait_inl(p_full, (ch0 + i) & 1, err))) break;
          // the first P.V of a unit overwrites O_h: the previous unit's
          // epilogue must have read it (the QKs above already overlap it)
          if (i == 0 && used > 0 && !(ok = mbar_wait_inl(o_free, (used - 1) & 1, err))) break;
          if (i == 0 && used > 0 && !two && !(ok = mbar_wait_inl(o_free + 1, (used - 1) & 1, err))) break;
          if (kFp8 && !(ok = mbar_wait_inl(v_full + s, (it >> 1) & 1, err))) break;
          tc_fence_after();
          pv(0, s, i > 0);
          if (!two) mma_commit(kv_empty + s);
          if (more) {
            if (!(ok = mbar_wait_inl(kv_full + s1, ((it + 1) >> 1) & 1, err))) break;
            tc_fence_after();
            qk(0, s1);
            if (kFp8 && !two) mma_commit(k_empty + s1);
            if (!two && i + 1 == n - 1) mma_commit(q_empty);
          } else {
            mma_commit(o_done);
          }
          if (!two) continue;
          // head 1
          if (!(ok = mbar_wait_inl(p_full + 1, (ch1 + i) & 1, err))) break;
          if (i == 0 && used > 0 && !(ok = mbar_wait_inl(o_free + 1, (used - 1) & 1, err))) break;
          tc_fence_after();
          pv(1, s, i > 0);
          mma_commit(kv_empty + s);
          if (more) {
            qk(1, s1);
            if (kFp8) mma_commit(k_empty + s1);
            if (i + 1 == n - 1) mma_commit(q_empty);
          } else {
            mma_commit(o_done + 1);
          }
        }
        ch0 += n;
        if (two) ch1 += n;
        kv_it += n;
        ++used;
      }
      mma_commit(drain);
      mbar_wait_inl(drain, 0, err);
    }
  } else if (warp < kSoftWarps) {
    // ----------------------------------------------------------- softmax
    setmaxnreg_inc<kSoftRegs>();
    // Each unit's row statistics go to the epilogue warps, which normalise
    // and store O while these warps go on to the next unit's blocks.
    const int h = warp >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + h * 128;
    const uint32_t o_addr = tmem + lane_base + 256 + h * D;
    int ch = 0;  // blocks of head h so far
    int kv_it = 0;  // blocks of either so far
    bool ok = true;
    for (int k = 0, ui = first_unit(); ui < n_units; ++k, ui += kSplit ? n_units : gridDim.x) {
      const UnitHdr& ls = lhdr(k);
      const int32_t* const ls_j = kOneKvHead && h == 1 ? lj1(k) : lj(k);  // a paired unit's heads: own blocks
      if (ok) ok = mbar_wait_inl(list_full + k % kListSlots, (k / kListSlots) & 1, err);
      ok = __all_sync(0xFFFFFFFFu, ok);
      const int n = ok ? ls.n : 0, nh = ok ? ls.nh : 0;
      const int rows = ls.rows, pos0 = ls.pos0;
      // FP8: the scores are q . k_code, scaled by k_scale of the unit's KV head
      float sl2 = kFp8 && !kBlk ? scale_log2 * k_scale[ls.g] : scale_log2;
      float log2_vs = 0.f, inv_vs = 1.f;
      const bool active = ok && h < nh;
      const int lg = kBlk ? ls.lg : 0;
      const bool row_ok = (r >> lg) < rows;
      const int qpos = pos0 + (r >> lg);
      float m = -INFINITY, l = 0.f;
      for (int i = 0; active && ok && i < n; ++i) {
        if (kBlk) {
          const float2 sc = scale_ring[(kv_it + i) % kScaleRing];
          sl2 = sc.x, log2_vs = sc.y, inv_vs = ex2_approx(-sc.y);
        }
        if (!(ok = mbar_wait_inl(s_full + h, (ch + i) & 1, err))) break;
        tc_fence_after();
        uint32_t sv[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, sv + c * 32);
        tmem_wait_ld();
        const int j = ls_j[i];
        const bool pad = kOneKvHead && j < 0;  // the shorter list of a paired unit: every key masked
        const bool need_mask = pad || (j * 128 + 127 > pos0) || (rows < 128);
        if (need_mask) {  // only diagonal / ragged blocks: -inf past the row's position
          const int limit = row_ok && !pad ? qpos - j * 128 : -1;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > limit) sv[c] = __float_as_uint(-INFINITY);
        }
        float mx;
        {  // four independent chains keep the max off the latency path
          float a0 = -INFINITY, a1 = -INFINITY, a2 = -INFINITY, a3 = -INFINITY;
#pragma unroll
          for (int c = 0; c < 128; c += 8) {
            a0 = fmax3(a0, __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
            a1 = fmax3(a1, __uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3]));
            a2 = fmax3(a2, __uint_as_float(sv[c + 4]), __uint_as_float(sv[c + 5]));
            a3 = fmax3(a3, __uint_as_float(sv[c + 6]), __uint_as_float(sv[c + 7]));
          }
          mx = fmax3(fmaxf(a0, a1), a2, a3);
        }
        // lazy rescaling: the reference max moves only when the row max grows
        // by more than 2^8, so probabilities stay below 256 and O is rescaled
        // rarely
        const float mx2 = kBlk ? fmaf(mx, sl2, log2_vs) : mx * sl2;
        const float m_new = mx2 > m + 8.f ? mx2 : m;
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = m_new == m ? 1.f : ex2_approx(m - m_use);
        const float shift = kBlk ? log2_vs - m_use : -m_use;
        float sum0 = 0.f, sum1 = 0.f, sum2 = 0.f, sum3 = 0.f;
        uint32_t pk[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          float x0, x1;
          ffma2(x0, x1, __uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1]), sl2, shift);
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          if (c & 1)
            fadd2(sum2, sum3, p0, p1);
          else
            fadd2(sum0, sum1, p0, p1);
          pk[c] = kFp8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
        }
        sum0 += sum2;
        sum1 += sum3;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st16(s_addr + c * 16, pk + c * 16);
        l = l * alpha + (kBlk ? (sum0 + sum1) * inv_vs : sum0 + sum1);
        // rescale O_h (written by P.V of the previous block, already complete
        // because the S_h MMA of this block was issued after it)
        // (P_h.V of the previous block is complete: the MMA thread issued
        // this block's S_h after it, and s_full covers every earlier MMA)
        if (i > 0 && __any_sync(0xFFFFFFFFu, alpha != 1.f)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_addr + c * 32, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32(o_addr + c * 32, ov);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + h);
        m = m_new;
      }
      // this head's statistics (buffer k % 2, reused once the epilogue has
      // read its contents from two units back)
      const int b = k & 1;
      UnitStats& st = stats[h * 2 + b];
      if (k >= 2 && ok) ok = mbar_wait_inl(stat_empty + h * 2 + b, ((k >> 1) - 1) & 1, err);
      ok = __all_sync(0xFFFFFFFFu, ok);
      st.m[r] = m;
      st.l[r] = l;
      if (quarter == 0 && lane == 0) {
        st.n = n;
        st.active = active ? 1 : 0;
        st.ok = ok ? 1 : 0;
        st.h0 = ls.h0;
        st.q_begin = ls.q_begin;
        st.rows = rows;
        st.g = ls.g;
        st.h_end = ls.h_end;
        st.lg = lg;
      }
      if (h < nh) ch += n;
      kv_it += n;
      // the list slot may be refilled (every warp arrives once per unit, active or not)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(stat_full + h * 2 + b);
        mbar_arrive(list_empty + k % kListSlots);
      }
    }
  } else if (warp >= kEpiWarp0) {
    // ---------------------------------------------------------- epilogue
    setmaxnreg_dec<kEpiRegs>();
    // Per unit, head 0 then head 1: wait for the softmax's statistics and
    // for the unit's last P.V, read O_h in 32-column chunks, release it to
    // the next unit's P.V, and write bf16 O = O_h / l (times v_scale for
    // FP8) and the natural-log LSE.  Full tiles of FP8 plans go through the
    // shared staging buffer and TMA tensor stores.
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    int od0 = 0, od1 = 0;  // units with blocks of head 0 / head 1 so far
    int ost_uses = 0;      // 64-column boxes staged so far
    bool ok = true;
    for (int k = 0, ui = first_unit(); ui < n_units; ++k, ui += kSplit ? n_units : gridDim.x) {
      const int b = k & 1;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const UnitStats& st = stats[h * 2 + b];
        if (ok) ok = mbar_wait_inl(stat_full + h * 2 + b, (k >> 1) & 1, err);
        ok = __all_sync(0xFFFFFFFFu, ok);
        const int n = st.n, rows = st.rows, q_begin = st.q_begin, h0 = st.h0, st_h_end = st.h_end;
        const int lg = kBlk ? st.lg : 0;
        const bool active = ok && st.active != 0;
        const bool unit_ok = ok && st.ok != 0;
        const float m = st.m[r], l = st.l[r];
        const float o_scale = kFp8 && !kBlk ? v_scale[st.g] : 1.f;
        __syncwarp();
        if (lane == 0) mbar_arrive(stat_empty + h * 2 + b);
        if (!active) {
          __syncwarp();
          if (lane == 0 && n > 0) mbar_arrive(o_free + h);
          continue;
        }
        const bool has_o = n > 0;
        if (has_o && ok) ok = mbar_wait_inl(o_done + h, (h == 0 ? od0++ : od1++) & 1, err);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        const uint32_t o_addr = tmem + lane_base + 256 + h * D;
        const float inv_l = l > 0.f ? o_scale / l : 0.f;
        const int head = h0 + (h << lg) + (r & ((1 << lg) - 1));
        const bool row_ok = (r >> lg) < rows && (!kBlk || head < st_h_end);
        const int64_t orow = static_cast<int64_t>(q_begin + (r >> lg)) * hq + head;
        const bool staged = kStageO && rows == 128;
        uint8_t* const ob = smem + L::kOOff + r * 128;
        uint4* const dst = reinterpret_cast<uint4*>(out + orow * D);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          if (has_o) {
            tmem_ld32(o_addr + c * 32, ov);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = 0u;
          }
          if (c == D / 32 - 1) {  // all of O_h is in registers: the next unit's P.V may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && has_o) mbar_arrive(o_free + h);
          }
          if (kSplit) {  // a part's O as it is, for the merge
#pragma unroll
            for (int e = 0; e < 8; ++e) part_o(smem, h, r, 8 * c + e) = *reinterpret_cast<const uint4*>(ov + 4 * e);
            continue;
          }
          // staged: one 64-column box at a time, once the previous box's
          // store has read the buffer
          if (staged && (c & 1) == 0 && ost_uses > 0 && ok) ok = mbar_wait_inl(ost_free, (ost_uses - 1) & 1, err);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t* x = ov + 8 * e;
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(x[0]) * inv_l, __uint_as_float(x[1]) * inv_l);
            w.y = pack_bf16x2(__uint_as_float(x[2]) * inv_l, __uint_as_float(x[3]) * inv_l);
            w.z = pack_bf16x2(__uint_as_float(x[4]) * inv_l, __uint_as_float(x[5]) * inv_l);
            w.w = pack_bf16x2(__uint_as_float(x[6]) * inv_l, __uint_as_float(x[7]) * inv_l);
            if (staged) {
              // the TMA box layout: 64-column chunks of 128-byte rows, 16-byte
              // units swizzled by row % 8
              const int unit = (c & 1) * 4 + e;
              *reinterpret_cast<uint4*>(ob + ((unit ^ (r & 7)) << 4)) = w;
            } else if (unit_ok && row_ok) {
              dst[c * 4 + e] = w;
            }
          }
          if (staged && (c & 1) == 1) {  // the box is complete: one thread stores it
            fence_async_shared();        // the TMA store reads it through the async proxy
            __syncwarp();
            if (lane == 0) mbar_arrive(ost_ready);
            if (quarter == 0 && lane == 0) {
              if (ok) ok = mbar_wait_inl(ost_ready, ost_uses & 1, err);
              if (ok && unit_ok) {
                tma_store_3d(&o_map, smem + L::kOOff, 64 * (c >> 1), h0 + h, q_begin);
                bulk_commit_group();
              }
              bulk_wait_group_read0();
              mbar_arrive(ost_free);
            }
            ++ost_uses;
          }
        }
        if (!kSplit && unit_ok && row_ok && lse != nullptr)
          lse[orow] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
    }
    if (kStageO && quarter == 0 && lane == 0) bulk_wait_group0();  // the stores are complete
  } else if (kFp8) {
    // -------------------------------------------------- FP8 converters
    setmaxnreg_dec<kWg2Regs>();
    // Thread ct of the two warps owns rows ct and ct + 64 of every K / V
    // block: it reads a row's 128 e4m3 codes (eight 16-byte units of the
    // swizzled upper half of the stage) before it writes any of the row's
    // f16 units, and the only f16 units that land in that upper half are the
    // same row's, so no other thread's codes are overwritten.
    const int ct = threadIdx.x - 32 * (kSoftWarps + 2);
    auto expand128 = [&](uint8_t* buf, int rows) {  // buf: one ring stage, 2 chunks x [128 rows][128 B] of f16
#pragma unroll 1
      for (int rr = 0; rr < 2; ++rr) {
        const int r = ct + 64 * rr, sw = r & 7;
        const uint8_t* raw = buf + 16384 + r * 128;
        uint4 u[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) u[c] = *reinterpret_cast<const uint4*>(raw + ((c ^ sw) << 4));
        if (kBlk && r >= rows) {  // behind the sequence's last key
#pragma unroll
          for (int c = 0; c < 8; ++c) u[c] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {  // codes of d in [16c, 16c + 16) -> two f16 units
          uint4 lo, hi;
          lo.x = e4m3x2_to_f16x2(u[c].x);
          lo.y = e4m3x2_to_f16x2(u[c].x >> 16);
          lo.z = e4m3x2_to_f16x2(u[c].y);
          lo.w = e4m3x2_to_f16x2(u[c].y >> 16);
          hi.x = e4m3x2_to_f16x2(u[c].z);
          hi.y = e4m3x2_to_f16x2(u[c].z >> 16);
          hi.z = e4m3x2_to_f16x2(u[c].w);
          hi.w = e4m3x2_to_f16x2(u[c].w >> 16);
          uint8_t* dst = buf + (c >> 2) * 16384 + r * 128;
          const int u0 = (c & 3) * 2;
          *reinterpret_cast<uint4*>(dst + ((u0 ^ sw) << 4)) = lo;
          *reinterpret_cast<uint4*>(dst + (((u0 + 1) ^ sw) << 4)) = hi;
        }
      }
    };
    // head_dim 64: a stage is one chunk of 64 f16 columns, its upper half the
    // 64-byte rows of codes, and the f16 rows from 64 on land on other rows'
    // codes: both warps have read all of them before either writes (a bounded
    // wait, so that one warp's timeout ends the other's too).
    uint32_t halves = 0;
    auto expand64 = [&](uint8_t* buf, int rows) {
      uint4 u[2][4];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int r = ct + 64 * rr;
        const uint8_t* raw = buf + 8192 + r * 64;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          u[rr][c] = *reinterpret_cast<const uint4*>(raw + ((c ^ ((r >> 1) & 3)) << 4));
          if (r >= rows) u[rr][c] = make_uint4(0u, 0u, 0u, 0u);  // behind the sequence's last key
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(conv_read);
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_inl(conv_read, halves++ & 1, err))) return false;
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int r = ct + 64 * rr, sw = r & 7;
        uint8_t* dst = buf + r * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 v = u[rr][c];
          *reinterpret_cast<uint4*>(dst + (((2 * c) ^ sw) << 4)) =
              make_uint4(e4m3x2_to_f16x2(v.x), e4m3x2_to_f16x2(v.x >> 16), e4m3x2_to_f16x2(v.y),
                         e4m3x2_to_f16x2(v.y >> 16));
          *reinterpret_cast<uint4*>(dst + (((2 * c + 1) ^ sw) << 4)) =
              make_uint4(e4m3x2_to_f16x2(v.z), e4m3x2_to_f16x2(v.z >> 16), e4m3x2_to_f16x2(v.w),
                         e4m3x2_to_f16x2(v.w >> 16));
        }
      }
      return true;
    };
    auto expand = [&](uint8_t* buf, int rows) {
      if constexpr (D == 64) return expand64(buf, rows);
      expand128(buf, rows);
      return true;
    };
    int kv_it = 0;
    bool ok = true;
    for (int k = 0, ui = first_unit(); ok && ui < n_units; ++k, ui += kSplit ? n_units : gridDim.x) {
      const UnitHdr& ls = lhdr(k);
      ok = mbar_wait_inl(list_full + k % kListSlots, (k / kListSlots) & 1, err);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      const int n = ls.n, nh = ls.nh, kv_len = ls.kv_len;
      const int32_t* const ls_j = lj(k);
      __syncwarp();
      if (!kBlk && lane == 0) mbar_arrive(list_empty + k % kListSlots);
      // Q of the unit's heads, bf16 -> f16 in place
      if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait_inl(q_full, k & 1, err)))) break;
      for (int hh = 0; hh < nh; ++hh) {
        uint4* qv = reinterpret_cast<uint4*>(q_s + hh * L::kTileBytes);
#pragma unroll 4
        for (int e = ct; e < L::kTileBytes / 16; e += 32 * kConvWarps) {
          uint4 v = qv[e];
          v.x = bf16x2_to_f16x2(v.x);
          v.y = bf16x2_to_f16x2(v.y);
          v.z = bf16x2_to_f16x2(v.z);
          v.w = bf16x2_to_f16x2(v.w);
          qv[e] = v;
        }
      }
      fence_async_shared();  // the MMAs read these through the async proxy
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
      for (int i = 0; i < n; ++i, ++kv_it) {
        const int s = kv_it % kStages;
        if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait_inl(raw_full + s, (kv_it / kStages) & 1, err)))) break;
        if (!(ok = expand(k_s + s * L::kTileBytes, 128))) break;
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full + s);
        if (!(ok = __all_sync(0xFFFFFFFFu, mbar_wait_inl(raw_v_full + s, (kv_it / kStages) & 1, err)))) break;
        if (!(ok = expand(v_s + s * L::kTileBytes, kBlk ? kv_len - ls_j[i] * 128 : 128))) break;
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_full + s);
      }
      if (kBlk && lane == 0) mbar_arrive(list_empty + k % kListSlots);  // read up to here
    }
  } else {
    setmaxnreg_dec<kWg2Regs>();  // warps 10-11 without FP8 K/V: idle
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
  if constexpr (kSplit) {
    cluster_sync();  // every part's O, m and l are in its shared memory
    if (warp < kSoftWarps) {
      // Part p merges rows p, p + parts, ... of the unit: first every row's
      // weights (where Q was), then its O, a chunk of all parts at a time.
      constexpr int kThreads = 32 * kSoftWarps, kMost = 8;
      const AttnUnit u = units[first_unit()];
      const TileInfo tl = tiles[u.tile];
      const int lg = u.lg;
      const int mine = ((tl.rows << lg) - part + parts - 1) / parts;  // rows 1..128, parts <= 8
      const int h_end = (u.g + 1) * (hq / hsel);
      auto head_of = [&](int h, int r) { return u.h0 + (h << lg) + (r & ((1 << lg) - 1)); };
      float* const wts = reinterpret_cast<float*>(q_s);       // [head * mine + row][kMost]
      for (int e = threadIdx.x; e < u.nh * mine; e += kThreads) {
        const int h = e >= mine, r = part + (e - h * mine) * parts;
        const uint32_t m_at = smem_u32(&stats[2 * h].m[r]), l_at = smem_u32(&stats[2 * h].l[r]);
        float m[kMost], l[kMost], mm = -INFINITY, sum = 0.f;
#pragma unroll
        for (int p = 0; p < kMost; ++p)
          if (p < parts) m[p] = ld_cluster_f1(m_at, p), l[p] = ld_cluster_f1(l_at, p);
#pragma unroll
        for (int p = 0; p < kMost; ++p)
          if (p < parts) mm = fmaxf(mm, m[p]);
#pragma unroll
        for (int p = 0; p < kMost; ++p)
          if (p < parts) {
            m[p] = m[p] == -INFINITY ? 0.f : ex2_approx(m[p] - mm);
            sum += l[p] * m[p];
          }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int p = 0; p < kMost; ++p)
          if (p < parts) wts[e * kMost + p] = m[p] * inv;
        if (lse != nullptr && head_of(h, r) < h_end)
          lse[static_cast<int64_t>(tl.q_begin + (r >> lg)) * hq + head_of(h, r)] =
              sum > 0.f ? (mm + log2f(sum)) * 0.69314718055994531f : -INFINITY;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
#pragma unroll 1
      for (int e = threadIdx.x; e < u.nh * mine * (D / 4); e += kThreads) {
        const int item = e / (D / 4), chunk = e % (D / 4);
        const int h = item >= mine, r = part + (item - h * mine) * parts;
        const uint32_t at = smem_u32(&part_o(smem, h, r, chunk));
        float4 op[kMost], o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int p = 0; p < kMost; ++p)
          if (p < parts) op[p] = ld_cluster_f4(at, p);
#pragma unroll
        for (int p = 0; p < kMost; ++p)
          if (p < parts) {
            const float w = wts[item * kMost + p];
            o.x += op[p].x * w, o.y += op[p].y * w, o.z += op[p].z * w, o.w += op[p].w * w;
          }
        if (head_of(h, r) < h_end)
          *reinterpret_cast<uint2*>(out + (static_cast<int64_t>(tl.q_begin + (r >> lg)) * hq + head_of(h, r)) * D +
                                    4 * chunk) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
      }
    }
    cluster_sync();  // nobody leaves while its part may be read
    if ((chain & kFollows) && threadIdx.x == 0) pdl_wait();
  }
}

}  // namespace

// Orders the units for the persistent grid, whose CTA c takes units c, c + grid,
// c + 2 grid, ...: heaviest first, each round's heaviest to the CTA with the
// least so far, and the last, partial round to the CTAs with the least of all
// (which become the first columns).  A unit visits at most min(num_valid_pages,
// topk) blocks; a block step of one head takes about 0.8 of one of two, and a
// unit about a step besides.  176 units (6 ragged sequences, three heads a
// group) on 152 SMs: 54 -> 44 us.  The lightest n_split units stay at the end
// for a launch of their own.
static void balance_units(const msa_plan_s* p, std::vector<AttnUnit>& us, int n_split = 0) {
  const int n = static_cast<int>(us.size()) - n_split, grid = std::min(n, p->num_sms);
  auto cost = [&](const AttnUnit& u) {
    return int64_t(std::min(p->tiles[u.tile].nvp, p->topk) + 1) * (u.nh == 2 ? 5 : 4);
  };
  std::stable_sort(us.begin(), us.end(), [&](const AttnUnit& a, const AttnUnit& b) { return cost(a) > cost(b); });
  if (grid == 0) return;
  std::vector<int64_t> load(grid, 0);
  std::vector<int> col(grid);
  for (int c = 0; c < grid; ++c) col[c] = c;
  std::vector<AttnUnit> out(us);
  std::vector<int> place(n);  // column of each unit
  auto by_load = [&](int a, int b) { return load[a] < load[b]; };
  for (int base = 0; base < n; base += grid) {
    std::stable_sort(col.begin(), col.end(), by_load);
    for (int i = 0; i < std::min(grid, n - base); ++i) {
      place[base + i] = col[i];
      load[col[i]] += cost(us[base + i]);
    }
  }
  // columns by rank in the last round, so that a partial one fills the first
  std::vector<int> label(grid);
  for (int i = 0; i < grid; ++i) label[col[i]] = i;
  for (int i = 0; i < n; ++i) out[i / grid * grid + label[place[i]]] = us[i];
  us.swap(out);
}

// Tiles of few rows (block scales): log2 of the heads of a group that go side by
// side into the 128 M rows, as many as fit, so that a block step serves them
// all; otherwise most of each product and of each softmax row would be padding.
// Measured (us), a head a tile -> packed:
//   32 x 4 rows, 64 / 8 heads, 16 blocks   274 -> 72.7
//   64 x 2 rows, 128 / 8 heads, 16 blocks 1037 -> 136
//   30 x 9 rows, 128 / 8 heads, 2 blocks   108 -> 22.1
//    1 x 4 rows, 64 / 8 heads, 16 blocks  20.3 -> 13.8
// Each tile its own number, as decode rows beside a chunk want it (64 / 8 heads, 16 blocks):
//   32 x 1 row + 512 rows                  308 -> 107
//   64 x 1 row + 2048 rows                 637 -> 240
//   12 x 1..400 rows, 32 / 4 heads         116 -> 84.9
static int pack_of(const msa_plan_s* p, const TileInfo& t) {
  int lg = 0;
  if (p->kv_dtype == MSA_KV_FP8_E4M3_BLOCK)
    while (lg < kMaxPack && (t.rows << (lg + 1)) <= 128 && (2 << lg) <= p->hq / p->hp) ++lg;
  return lg;
}
static int slots_of(int heads, int lg) { return (heads + (1 << lg) - 1) >> lg; }

// Heads a unit, the units to split, the CTAs that share each of those, and the
// time that takes, estimated (block scales; us), without the tiles of `apart` rows or
// fewer.
//
// Two heads share a block's K and V and overlap each other's softmax; with an
// SM for every head, a head alone is done sooner (512 rows x 32 heads, topk 16:
// e4m3 38.0 us in pairs, 32.6 alone; bf16 34.4, 28.8).  Block-scaled plans also
// share a unit's blocks out over a cluster while each of its CTAs has an SM: all
// units, or those that a last, short round would be left with, in a launch of
// their own.  A block step takes about 1.65 us for a head and 1.78 for two (0.35
// more where no other unit reads the same blocks, which then come from HBM), a
// unit 6 besides, the merge 3 and a second launch 6.  Clusters of 8 are not
// placed as densely as the SMs would allow: 15 run at once.  The times are those
// of head_dim 128 and stand for 64 as well, which has shorter steps; the
// longest unit's blocks stand for every unit's.
// Measured (us; heads a unit / parts):
//   rows x heads, blocks     1/1    1/2    1/4    1/8    2/1    2/2    2/4
//     128 x 32, 16          33.8   24.4  [17.9]  41.7   38.3   29.2   21.1
//     512 x 32, 16          34.4   48.5   67.5    126   39.0  [30.1]  42.9
//       2 x 64, 16          39.2   25.3   33.3   61.8   42.4   27.1  [20.0]
//     300 x 4, 24           55.0   33.5   21.3  [16.4]  58.7   36.5   24.6
//     700 x 12, 9           24.5  [20.0]  31.3   69.2   27.7   24.1   30.9
//     100 x 8, 64            139   76.7   43.6  [27.3]   144   81.3   47.2
// 160 pairs on 152 SMs, the last 8 split: 16 blocks 84.5 -> 68.0, 64 292 -> 196.
struct UnitShape {
  double us;
  int heads;
  int64_t split;
  int parts;
};
static UnitShape unit_shape(const msa_plan_s* p, int apart) {
  const int sms = p->num_sms;
  const int grp = p->hq / p->hp;
  if (p->kv_dtype != MSA_KV_FP8_E4M3_BLOCK) return {0.0, int64_t(p->n_tiles) * p->hq <= sms ? 1 : 2, 0, 1};
  int blocks = 1;
  for (const TileInfo& t : p->tiles)
    if (t.rows > apart) blocks = std::max(blocks, std::min(t.nvp, p->topk));
  UnitShape best{1e30, 2, 0, 1};
  for (int heads = 2; heads >= 1; --heads) {
    int64_t units = 0, sets = 0;
    for (const TileInfo& t : p->tiles)
      if (t.rows > apart) {
        units += int64_t(p->hp) * ((slots_of(grp, pack_of(p, t)) + heads - 1) / heads);
        sets += p->hp;
      }
    const int64_t rounds = units / sms;
    const double step = (heads == 2 ? 1.78 : 1.65) + (units == sets ? 0.35 : 0.0), unit = blocks * step + 6;
    const int64_t rest = units - rounds * sms;
    auto take = [&](double us, int64_t split, int parts) {
      if (us < best.us) best = {us, heads, split, parts};
    };
    // an odd head beside pairs fills the rounds better than heads alone
    take((rounds + (rest > 0)) * unit * (heads == 1 && units > sms ? 1.1 : 1.0), 0, 1);
    for (int parts = 2; parts <= 8 && parts <= blocks && rest > 0; parts *= 2)
      if (rest * parts <= (parts < 8 ? sms - 8 : sms * 3 / 4))
        take(rounds * unit + (rounds > 0 ? 6 : 0) + (blocks + parts - 1) / parts * step + 9, rest, parts);
  }
  return best;
}

// Estimated time of the decode kernel for a batch's tiles of `apart` rows or
// fewer, in parts of up to 16 (row, head) columns: its ramp and the K and V bytes
// at the rate it reaches with one tile of 8 columns or with two.  None: 0.
static double rows_us(const msa_plan_s* p, int apart) {
  const int grp = p->hq / p->hp, most = 16 / grp;
  int64_t bytes = 0, blocks = 0;
  int columns = 0;
  for (const TileInfo& t : p->tiles)
    if (t.rows <= apart) {
      const int64_t n = std::min(t.nvp, p->topk);
      bytes += n * ((t.rows + most - 1) / most) * p->hp * 2 * 128 * p->d;
      blocks = std::max(blocks, n), columns = std::max(columns, std::min(t.rows, most) * grp);
    }
  return bytes > 0 ? 6 + bytes / (columns > 8 ? 4.7e6 : 6.4e6) + 0.03 * blocks : 0.0;
}

void attn_plan_tables(msa_plan_s* p, std::vector<int32_t>& aux) {
  // a unit: (tile, proxy head g, a pair of the query heads that use g's
  // blocks); with one proxy head per GQA group g is the group
  std::vector<AttnUnit> us;
  const int grp = p->hq / p->hp;
  UnitShape shape = unit_shape(p, 0);
  // block scales: tiles of few rows in a launch of the decode kernel where that
  // is done sooner.  Measured (us, 16 blocks; all as tiles -> so):
  //   32 x 1 + 512 rows, 64 / 8 heads   107 -> 66.0      64 x 4, 32 / 8   136 -> 70.6
  //   64 x 1 + 2048 rows, 64 / 8        240 -> 203       16 x 4, 32 / 8  39.9 -> 16.7
  //   32 x 2 rows, 64 / 8              73.4 -> 35.5      16 x 8, 32 / 8  39.8 -> 31.7
  //   32 x 4 rows, 64 / 8 (two parts)  73.2 -> 66.3       8 x 2, 64 / 8  25.9 -> 12.7
  // and where it is not: 16 x 4 rows, 64 / 4 (four parts) 26.8, 31.0; 30 x 9 rows,
  // 128 / 8, 2 blocks 21.9, 89; 4 x 1 + 128 rows, 16 / 2 17.4, 25.9.  That launch
  // comes last and starts as the others' SMs fall idle (kFollows): 6 ragged chunks,
  // 12 / 4 heads, 9 blocks, 40.9 -> 32.5 us.
  const int most = 16 / grp;  // rows a part of those
  int apart = 0;
  std::vector<int32_t> parts;  // two words each
  if (p->kv_dtype == MSA_KV_FP8_E4M3_BLOCK && !p->decode && most > 0) {
    double best = shape.us;
    for (int rows = 1; rows <= 16; ++rows) {
      const UnitShape rest = unit_shape(p, rows);
      const double us = rows_us(p, rows) + (rest.us > 0 ? rest.us + 2 : 0);
      if (us < best) best = us, apart = rows, shape = rest;
    }
    for (int t = 0; t < p->n_tiles; ++t)
      for (int r = 0; p->tiles[t].rows <= apart && r < p->tiles[t].rows; r += most) {
        const int n = std::min(most, p->tiles[t].rows - r);
        parts.insert(parts.end(), {t, r | n << 16});
        p->row_part_heads = std::max(p->row_part_heads, n * grp);
      }
  }
  p->attn_split = static_cast<int32_t>(shape.split);
  p->attn_parts = shape.parts;
  aux.resize((aux.size() + 3) & ~size_t(3));
  p->row_parts_off = static_cast<int64_t>(aux.size());
  p->n_row_parts = static_cast<int32_t>(parts.size() / 2);
  aux.insert(aux.end(), parts.begin(), parts.end());
  aux.resize((aux.size() + 3) & ~size_t(3));
  const int pair = shape.heads;
  for (int t = 0; t < p->n_tiles; ++t) {
    if (p->tiles[t].rows <= apart) continue;
    const int lg = pack_of(p, p->tiles[t]), slots = slots_of(grp, lg);  // heads, or groups of heads side by side
    p->attn_packs |= 1 << lg;
    for (int g = 0; g < p->hp; ++g)
      for (int h = 0; h < slots; h += pair)
        us.push_back(AttnUnit{t, g, g * grp + (h << lg), static_cast<int16_t>(std::min(pair, slots - h)),
                              static_cast<int16_t>(lg)});
  }
  balance_units(p, us, p->attn_split);
  p->attn_units_off = static_cast<int64_t>(aux.size());
  p->n_attn_units = static_cast<int32_t>(us.size());
  const int32_t* raw = reinterpret_cast<const int32_t*>(us.data());
  aux.insert(aux.end(), raw, raw + us.size() * 4);
  // the proxy softmax of the backward: proxy heads g and g + 1 of a tile in
  // one unit, each over its own blocks (the two heads' softmaxes overlap each
  // other's products)
  std::vector<AttnUnit> ps;
  for (int t = 0; t < p->n_tiles; ++t)
    for (int g = 0; g < p->hp; g += 2) ps.push_back(AttnUnit{t, g, g, static_cast<int16_t>(std::min(2, p->hp - g)), 0});
  balance_units(p, ps);
  p->proxy_attn_units_off = static_cast<int64_t>(aux.size());
  p->n_proxy_attn_units = static_cast<int32_t>(ps.size());
  raw = reinterpret_cast<const int32_t*>(ps.data());
  aux.insert(aux.end(), raw, raw + ps.size() * 4);
}

namespace {

constexpr int kMaxSmem = 232448;  // 227 KB of dynamic shared memory per CTA

// Launches one instantiation: with O staged through shared memory (full
// tiles stored by TMA) for FP8 K/V when the list slots for this topk leave
// room for the staging buffer, else with per-thread stores.  Measured at
// S=32768: FP8 973 -> 1019 TFLOP/s staged; bf16 0.808 -> 0.826 ms staged,
// so bf16 keeps the per-thread stores.
// The register split above assumes the kernel is launched at exactly
// kLaunchRegs a thread; any other count would leave an increase waiting, so
// such a build is not launched.
template <typename K>
cudaError_t check_launch_regs(K kern) {
  cudaFuncAttributes a;
  const cudaError_t e = cudaFuncGetAttributes(&a, kern);
  if (e != cudaSuccess) return e;
  return a.numRegs == kLaunchRegs ? cudaSuccess : cudaErrorInvalidConfiguration;
}

template <int D, bool kOneKvHead, bool kFp8, bool kBlk = false>
cudaError_t launch_attn_variant(dim3 grid, cudaStream_t st, const QueryMaps<kBlk>& qm, const CUtensorMap& km,
                                const CUtensorMap& vm, const CUtensorMap& om, int32_t topk, const AttnUnit* units,
                                int32_t n_units, const TileInfo* tiles, const int32_t* idx,
                                const int32_t* kv_indices, int64_t num_pages, __nv_bfloat16* o, float* lse,
                                int32_t hq, int32_t hsel, int32_t kv_div, float scale_log2, const float* k_scale,
                                const float* v_scale, uint32_t* err, int parts = 1, int chain = 0) {
  const int cap = (topk + 3) & ~3;
  if constexpr (kFp8) {
    const int staged = AttnSmem<D, true, kOneKvHead ? 2 : 1, kBlk>::bytes(cap) + 1024;
    if (staged <= kMaxSmem && parts == 1) {
      auto kern = attn_fwd_kernel<D, kOneKvHead, kFp8, true, kBlk>;
      if constexpr (kBlk)
        if (chain & kLeads) kern = attn_fwd_kernel<D, kOneKvHead, kFp8, true, true, false, true>;
      if (const cudaError_t e = check_launch_regs(kern)) return e;
      // the limit is the function's, for every host thread: always the most of any topk
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
      return launch_pdl_cluster(kern, grid, 1, dim3(kAttnThreads), staged, st, qm, km, vm, om, cap, units, n_units,
                                tiles, idx, kv_indices, num_pages, o, lse, hq, hsel, kv_div, topk, scale_log2, k_scale,
                                v_scale, 1, err, chain);
    }
  }
  const int plain = AttnSmem<D, false, kOneKvHead ? 2 : 1, kBlk>::bytes(kMaxTopk) + 1024;
  auto kern = attn_fwd_kernel<D, kOneKvHead, kFp8, false, kBlk>;
  if constexpr (kBlk) {
    if (parts > 1)
      kern = attn_fwd_kernel<D, kOneKvHead, kFp8, false, true, true>;
    else if (chain & kLeads)
      kern = attn_fwd_kernel<D, kOneKvHead, kFp8, false, true, false, true>;
  }
  if (const cudaError_t e = check_launch_regs(kern)) return e;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, plain);
  return launch_pdl_cluster(kern, grid, parts, dim3(kAttnThreads), plain, st, qm, km, vm, om, cap, units, n_units,
                            tiles, idx, kv_indices, num_pages, o, lse, hq, hsel, kv_div, topk, scale_log2, k_scale,
                            v_scale, parts, err, chain);
}

// [total_q, heads, D] bf16 rows as 3-D boxes of 64 columns x 1 head x 128 rows, 128-byte swizzle
// (pack_log2: 2^pack_log2 heads x 128 / 2^pack_log2 rows)
bool rows_map(CUtensorMap* m, const void* base, int d, int heads, int64_t total_q, int pack_log2 = 0) {
  const uint64_t dims[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(heads), static_cast<uint64_t>(total_q)};
  const uint64_t str[2] = {static_cast<uint64_t>(d) * 2, static_cast<uint64_t>(heads) * d * 2};
  const uint32_t box[3] = {64, 1u << pack_log2, 128u >> pack_log2};
  return encode_tensor_map(m, 3, base, dims, str, box, 1, 128);
}

}  // namespace

msa_status launch_attn_prefill(const msa_plan_s* p, const void* q, const void* k_pages, const void* v_pages,
                               const int32_t* kv_indices, const int32_t* idx, const float* k_scale,
                               const float* v_scale, void* out, float* lse, cudaStream_t st) {
  if (p->topk > kMaxTopk) return set_error(MSA_ERR_UNSUPPORTED, "msa_sparse_attn: topk above 1024");
  const bool fp8 = p->kv_dtype != MSA_KV_BF16;
  if (p->kv_dtype == MSA_KV_FP8_E4M3 && p->d != 128)
    return set_error(MSA_ERR_UNSUPPORTED, "msa_sparse_attn: FP8 K/V prefill needs head_dim 128");
  QueryMaps<true> qms{};  // the launch copies those of packs no unit has, too
  QueryMaps<false> qm;
  CUtensorMap km, vm, om;
  const int kv_elem = fp8 ? 1 : 2;
  const uint64_t kdims[2] = {static_cast<uint64_t>(p->d), static_cast<uint64_t>(p->num_pages) * p->hkv * 128};
  const uint64_t kstr[1] = {static_cast<uint64_t>(p->d) * kv_elem};
  // bf16: 64-column boxes (128 B rows); e4m3: whole rows of codes
  const uint32_t kbox[2] = {fp8 ? static_cast<uint32_t>(p->d) : 64u, 128};
  const int kswz = fp8 ? p->d : 128;
  const bool blk = p->kv_dtype == MSA_KV_FP8_E4M3_BLOCK;
  bool maps = blk || rows_map(&qm.by_lg[0], q, p->d, p->hq, p->total_q);
  for (int lg = 0; blk && lg <= kMaxPack; ++lg)
    if (p->attn_packs >> lg & 1) maps = maps && rows_map(&qms.by_lg[lg], q, p->d, p->hq, p->total_q, lg);
  if (!maps || !rows_map(&om, out, p->d, p->hq, p->total_q) ||
      !encode_tensor_map(&km, 2, k_pages, kdims, kstr, kbox, fp8 ? 0 : 1, kswz) ||
      !encode_tensor_map(&vm, 2, v_pages, kdims, kstr, kbox, fp8 ? 0 : 1, kswz))
    return set_error(MSA_ERR_CUDA, "msa_sparse_attn: tensor map encoding failed");
  const AttnUnit* units = reinterpret_cast<const AttnUnit*>(p->aux_d + p->attn_units_off);
  const float scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(p->d));
  auto* o = static_cast<__nv_bfloat16*>(out);
  const dim3 grid(std::min(p->n_attn_units, p->num_sms));  // persistent: one CTA per SM
  const int kv_div = p->hp / p->hkv;
  cudaError_t e;
  if (blk) {
    const auto launch = p->d == 128 ? launch_attn_variant<128, false, true, true>
                                    : launch_attn_variant<64, false, true, true>;
    const int whole = p->n_attn_units - p->attn_split;
    auto run = [&](int ctas, const AttnUnit* first, int n, int parts, int chain) {
      return launch(dim3(ctas), st, qms, km, vm, om, p->topk, first, n, p->tiles_d, idx, kv_indices, p->num_pages, o, lse,
                    p->hq, p->hp, kv_div, scale_log2, k_scale, v_scale, p->err_d, parts, chain);
    };
    e = whole > 0 ? run(std::min(whole, p->num_sms), units, whole, 1, p->attn_split > 0 || p->n_row_parts > 0 ? kLeads : 0)
                  : cudaSuccess;
    if (e == cudaSuccess && p->attn_split > 0)
      e = run(p->attn_split * p->attn_parts, units + whole, p->attn_split, p->attn_parts,
              (whole > 0 ? kFollows : 0) | (p->n_row_parts > 0 ? kLeads : 0));
  } else if (fp8)
    e = launch_attn_variant<128, false, true>(grid, st, qm, km, vm, om, p->topk, units, p->n_attn_units, p->tiles_d,
                                              idx, kv_indices, p->num_pages, o, lse, p->hq, p->hp, kv_div, scale_log2,
                                              k_scale, v_scale, p->err_d);
  else if (p->d == 128)
    e = launch_attn_variant<128, false, false>(grid, st, qm, km, vm, om, p->topk, units, p->n_attn_units, p->tiles_d,
                                               idx, kv_indices, p->num_pages, o, lse, p->hq, p->hp, kv_div,
                                               scale_log2, nullptr, nullptr, p->err_d);
  else
    e = launch_attn_variant<64, false, false>(grid, st, qm, km, vm, om, p->topk, units, p->n_attn_units, p->tiles_d,
                                              idx, kv_indices, p->num_pages, o, lse, p->hq, p->hp, kv_div, scale_log2,
                                              nullptr, nullptr, p->err_d);
  return cuda_check(e, "msa_sparse_attn: prefill launch");
}

// The proxy softmax of the backward (the KL term's p_proxy): for proxy head g
// of each tile, over group g's cached visible keys, Op = sum_k p(k) pk[k]
// and its natural-log LSE, with scores pq.pk/sqrt(dp).  It is the forward
// above with pq as the queries, the one shared proxy K head as both keys and
// values, and one head per unit.  Op: bf16 [total_q, Hp, 64]; lse: fp32
// [total_q, Hp].
msa_status launch_proxy_softmax(const msa_plan_s* p, const void* pq, const void* pk_pages, const int32_t* kv_indices,
                                const int32_t* idx, void* op, float* lse, cudaStream_t st) {
  if (p->topk > kMaxTopk) return set_error(MSA_ERR_UNSUPPORTED, "msa_sparse_attn_bwd: topk above 1024");
  QueryMaps<false> qm;
  CUtensorMap km, om;
  // pq and pk at dp = 32 are read as 64-column boxes whose upper half lies
  // past the tensor's edge: TMA fills it with zeros, so the dp = 64 kernel
  // computes the same scores and an Op whose columns [dp, 64) are zero
  const uint64_t kdims[2] = {static_cast<uint64_t>(p->dp), static_cast<uint64_t>(p->num_pages) * 128};
  const uint64_t kstr[1] = {static_cast<uint64_t>(p->dp) * 2};
  const uint32_t kbox[2] = {64, 128};
  if (!rows_map(&qm.by_lg[0], pq, p->dp, p->hp, p->total_q) || !rows_map(&om, op, 64, p->hp, p->total_q) ||
      !encode_tensor_map(&km, 2, pk_pages, kdims, kstr, kbox, 1, 128))
    return set_error(MSA_ERR_CUDA, "msa_sparse_attn_bwd: tensor map encoding failed");
  const AttnUnit* units = reinterpret_cast<const AttnUnit*>(p->aux_d + p->proxy_attn_units_off);
  const float scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(p->dp));
  const dim3 grid(std::min(p->n_proxy_attn_units, p->num_sms));
  return cuda_check(launch_attn_variant<64, true, false>(grid, st, qm, km, km, om, p->topk, units,
                                                          p->n_proxy_attn_units, p->tiles_d, idx, kv_indices,
                                                          p->num_pages, static_cast<__nv_bfloat16*>(op), lse, p->hp,
                                                          p->hp, p->hp, scale_log2, nullptr, nullptr, p->err_d),
                    "msa_sparse_attn_bwd: proxy softmax launch");
}

}  // namespace msa
