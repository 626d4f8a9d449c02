// Stage 3 (decode), one CTA or one cluster per (sequence, group) row: paged
// sparse attention with FP8 e4m3 K/V ("MiniMax-AI/MSA" README, section
// "Stacks": paged FP8 decode), the same arithmetic as decode_kernel in
// decode.cu: softmax over the selected blocks' keys of
// q.(k_code*k_scale)/sqrt(d), out = P.(v_code*v_scale).
//
// Every warp streams its own units (kKeys keys of K and of V of one selected
// block) through a private buffer and keeps its own online-softmax state; the
// warps' states are merged once, at the end of the row.  With two CTAs per SM
// that is 16 independent warps per SM, each with loads in flight, and no
// producer warp or per-block CTA barrier.  Unit u of the row (slot u / kParts
// of kv_block_indexes, keys kKeys (u % kParts) ...) goes to warp u % W of the
// row's W warps.  K and V have a barrier each: the next unit's K is on its way
// from the moment this unit's logits are done, its V from the end of P.V.
//
// Per unit, on mma.sync (f16 in, f32 out), exactly as decode_kernel:
//   S^T = K . q^T     M = kKeys keys, N = 8 NT heads, K = d (e4m3 -> f16 in registers)
//   O^T += V^T . P^T  M = d,  N = 8 NT heads, K = kKeys keys (P^T by movmatrix)
// with d permuted so that every shared-memory read is one conflict-free word.
//
// kBlk: one scale for each (page, KV head) (BlockScale in msa_internal.h).  A
// unit lies in one page, so its scales are three numbers a warp broadcasts
// with the unit; they cost one fused add and one multiply a unit and thread.
// Units wholly behind the query position, or on a page outside the pool, are
// not loaded, and V rows behind the position are zeroed in shared memory (their
// bytes were never written, and 0 * NaN would reach the output).
//
// Few rows (kBlk): a row's warps are the warps of a cluster of cs CTAs, whose
// merged states cross over distributed shared memory, with neither partials
// in global memory nor a serial merge by the row's last CTA.
//
// Bound by HBM from about 256 rows on: 32 sequences x 16 blocks x 8 KV heads
// (135 MB) take 25.9 us, 5.2 TB/s, of which the ramp (page table, scales and
// first loads, then the merge) is about 5 us.  With few rows it is the same
// ramp alone: 6.9 us for one sequence.
#include "msa_internal.h"
#include "ptx.cuh"

#include <cuda_fp16.h>


namespace msa {
namespace {

// a unit is kKeys keys of one selected block (K and V), streamed by one warp
// through a private buffer; kWsWarps warps per CTA, two CTAs per SM.
// Measured at 32 x 131072 (keys, stages, warps): (64,1,6) 29.9 us,
// (32,2,6) 30.4, (64,2,3) 31.0, (64,1,4) 29.7, (32,1,12) 35.5 (spills),
// (32,1,8) 28.9: 16 warps per SM and the same unit count for every warp.
constexpr int kKeys = 32;
constexpr int kWsWarps = 8;
constexpr int kWsThreads = 32 * kWsWarps;
constexpr int kParts = 128 / kKeys;             // units per block
constexpr int kMT = kKeys / 16;                 // 16-key m-tiles of a unit
constexpr int kMaxStaticTopk = (32 * kWsWarps) / kParts;

template <int D, int NT>
struct WsSmem {
  static constexpr int kHeads = 8 * NT;
  static constexpr int kPartBytes = kKeys * D;      // K (or V) bytes of one unit
  static constexpr int kBufBytes = 2 * kPartBytes;  // one warp's buffer: K part | V part
  static constexpr int kD = D;
  static_assert(kBufBytes >= kHeads * kD * 4, "a warp's O fits its buffer");
  static constexpr int kBufOff = 0;
  static constexpr int kCtaOff = kWsWarps * kBufBytes;            // the CTA's merged O, for its cluster
  static constexpr int kMlOff = kCtaOff + kHeads * kD * 4;        // (m, l) of each warp's heads, then the CTA's
  static constexpr int kBarOff = kMlOff + (kWsWarps + 1) * kHeads * 8;
  static constexpr int kBytes = kBarOff + 16 * kWsWarps;
};

// byte offset of (row, byte col) in a tile of D-byte rows written by TMA with
// D-byte swizzle: within a 128-byte line the 16-byte chunk index is XORed with
// the line's (D = 128) or the line pair's (D = 64) number.
template <int D>
__device__ __forceinline__ uint32_t swz(int row, int col) {
  if (D == 128) return row * 128 + ((((col >> 4) ^ row) & 7) << 4) + (col & 15);
  return row * 64 + ((((col >> 4) ^ (row >> 1)) & 3) << 4) + (col & 15);
}

// Merge of n states (m, l, O) of one head and four dims: stable in the log2
// domain, in the order given.
struct Merged {
  float m, l;
  float4 o;
};

template <bool kBlk, int kD, int NT, bool kFew>
__global__ void __launch_bounds__(kWsThreads, NT == 1 ? 2 : 1)
    decode_ws_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                     const __nv_bfloat16* __restrict__ q, const TileInfo* __restrict__ tiles,
                     const int2* __restrict__ part_list, const int32_t* __restrict__ idx, const int32_t* __restrict__ kv_indices, int64_t num_pages,
                     const float* __restrict__ k_scale, const float* __restrict__ v_scale,
                     __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int32_t hq, int32_t hsel,
                     int32_t kv_div, int32_t topk, int32_t cs, float scale_log2, int32_t chain, uint32_t* err) {
  if (kFew && (chain & kFollows))
    fence_gpu();
  else
    pdl_wait();
  using L = WsSmem<kD, NT>;
  constexpr int kPartBytes = L::kPartBytes, kBufBytes = L::kBufBytes, kMD = kD / 16;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // row = (sequence, proxy head g): the G = hq / hsel query heads of g over
  // g's blocks of KV head g / kv_div; CTA `rank` of the row's cs.  kFew: tiles of
  // few rows of a batch that has others too, part_list[] = (tile, first row |
  // rows << 16), rows * G <= 8 NT; "head" h is then head h % G of row h / G
  const int row = blockIdx.x / cs, rank = blockIdx.x % cs;
  const int g = row % hsel, G = hq / hsel;
  int t = row / hsel, first = 0, H = G;
  if (kFew) {
    const int2 part = part_list[t];
    t = part.x, first = part.y & 0xFFFF, H = G * (part.y >> 16);
  }
  const int hkv = hsel / kv_div, kvh = g / kv_div;
  const TileInfo tl = tiles[t];
  const int q_begin = tl.q_begin + first;
  uint8_t* buf = smem + L::kBufOff + warp * kBufBytes;
  uint64_t* bar_k = reinterpret_cast<uint64_t*>(smem + L::kBarOff) + 2 * warp;
  uint64_t* bar_v = bar_k + 1;
  if (lane == 0) {
    prefetch_tmap(&k_map);
    prefetch_tmap(&v_map);
    mbar_init(bar_k, 1);
    mbar_init(bar_v, 1);
    fence_mbar_init();
  }
  __syncwarp();

  // of the first query row and of the last
  const int qpos = tl.pos0 + first, last = kFew ? qpos + H / G - 1 : qpos;
  auto row_of = [&](int h) { return kFew ? h / G : 0; };
  auto head_of = [&](int h) { return kFew ? h % G : h; };
  const int n_units = kParts * topk;
  const int W = kWsWarps * cs, gw = rank * kWsWarps + warp;
  const int my_n = n_units > gw ? (n_units - gw + W - 1) / W : 0;
  int ukey = -1, urow = 0, n_valid = 0;
  // the next 32 of this warp's units gw, gw + W, ...: each lane looks up one;
  // the valid ones move to the low lanes (first key position, page row)
  auto fetch = [&](int base) {
    ukey = -1;
    if (base + lane < my_n) {
      const int u = gw + (base + lane) * W;
      const int j = idx[(static_cast<int64_t>(t) * hsel + g) * topk + u / kParts];
      if (j >= tl.nvp) {
        atomicOr(err, kErrDeviceCheck);
      } else if (j >= 0) {
        int64_t page = kv_indices[tl.page_base + j];
        const bool in_pool = page >= 0 && page < num_pages;
        if (!in_pool) {
          atomicOr(err, kErrDeviceCheck);
          page = 0;
        }
        ukey = j * 128 + (u % kParts) * kKeys;
        urow = static_cast<int>((page * hkv + kvh) * 128 + (u % kParts) * kKeys);
        if (kBlk && (ukey > last || !in_pool)) ukey = -1;
      }
    }
    // compact the valid units to the low lanes (padding slots load nothing)
    const unsigned vmask = __ballot_sync(0xFFFFFFFFu, ukey >= 0);
    n_valid = __popc(vmask);
    if (vmask & (vmask + 1)) {  // not the low lanes already
      unsigned rest = vmask;
      for (int k = 0; k < lane && k < n_valid; ++k) rest &= rest - 1;
      const int src = rest ? __ffs(rest) - 1 : 0;  // lane holding the (lane+1)-th valid unit
      ukey = __shfl_sync(0xFFFFFFFFu, ukey, src);
      urow = __shfl_sync(0xFFFFFFFFu, urow, src);
    }
  };
  auto load = [&](const CUtensorMap* map, uint64_t* bar, uint8_t* dst, int i) {
    const int r = __shfl_sync(0xFFFFFFFFu, urow, i);
    if (lane == 0) {
      mbar_expect_tx(bar, kPartBytes);
      tma_load_2d(dst, map, bar, 0, r);
    }
  };
  fetch(0);
  if (n_valid > 0) {
    load(&k_map, bar_k, buf, 0);
    load(&v_map, bar_v, buf + kPartBytes, 0);
  }

  // q^T fragments: head gi + 8 nt of the group, d = 16 kc + 4 t4 + {0,1} | {2,3}
  const int gi = lane >> 2, t4 = lane & 3;
  uint32_t qf[NT][kD / 16][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int hl = gi + 8 * nt;
    const __nv_bfloat16* qr = q + (static_cast<int64_t>(q_begin + row_of(hl)) * hq + g * G + head_of(hl)) * kD;
#pragma unroll
    for (int kc = 0; kc < kD / 16; ++kc) {
      if (hl < H) {
        const uint2 v = *reinterpret_cast<const uint2*>(qr + kc * 16 + 4 * t4);
        qf[nt][kc][0] = bf16x2_to_f16x2(v.x);  // beyond f16 saturating, as the prefill kernel has it
        qf[nt][kc][1] = bf16x2_to_f16x2(v.y);
      } else {
        qf[nt][kc][0] = qf[nt][kc][1] = 0u;
      }
    }
  }
  float sl2 = kBlk ? 0.f : scale_log2 * k_scale[kvh];
  float log2_vs = 0.f, inv_vs = 1.f;
  int qp[NT][2];  // positions of this thread's columns
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) qp[nt][c] = qpos + row_of(8 * nt + 2 * t4 + c);
  float m[NT][2], l[NT][2], oacc[kMD][NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int md = 0; md < kMD; ++md) oacc[md][nt][0] = oacc[md][nt][1] = oacc[md][nt][2] = oacc[md][nt][3] = 0.f;
  }
  const uint32_t kb = smem_u32(buf), vb = kb + kPartBytes;
  bool ok = true;
  uint32_t phase = 0;
  for (int base = 0; ok && base < my_n; base += 32) {
    if (base > 0) {
      fetch(base);
      if (n_valid > 0) {
        load(&k_map, bar_k, buf, 0);
        load(&v_map, bar_v, buf + kPartBytes, 0);
      }
    }
    BlockScale ubs{};
    if (kBlk && lane < n_valid) {
      ubs = block_scale_of(k_scale[urow >> 7], v_scale[urow >> 7]);
      ubs.ks *= scale_log2;
    }
    for (int i = 0; ok && i < n_valid; ++i, phase ^= 1) {
      const int key0 = __shfl_sync(0xFFFFFFFFu, ukey, i);
      if (kBlk) {
        sl2 = __shfl_sync(0xFFFFFFFFu, ubs.ks, i);
        log2_vs = __shfl_sync(0xFFFFFFFFu, ubs.log2_vs, i);
        inv_vs = __shfl_sync(0xFFFFFFFFu, ubs.inv_vs, i);
      }
      if (!(ok = mbar_wait(bar_k, phase, err))) break;

      // S^T for the unit's keys
      float sacc[kMT][NT][4];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        const int ra = 16 * mt + gi, rb = ra + 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sacc[mt][nt][0] = sacc[mt][nt][1] = sacc[mt][nt][2] = sacc[mt][nt][3] = 0.f;
#pragma unroll
        for (int kc = 0; kc < kD / 16; ++kc) {
          const uint32_t wa = lds32(kb + swz<kD>(ra, kc * 16 + 4 * t4));
          const uint32_t wb = lds32(kb + swz<kD>(rb, kc * 16 + 4 * t4));
          const uint32_t a0 = e4m3x2_to_f16x2(wa), a1 = e4m3x2_to_f16x2(wb);
          const uint32_t a2 = e4m3x2_to_f16x2(wa >> 16), a3 = e4m3x2_to_f16x2(wb >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16(sacc[mt][nt], a0, a1, a2, a3, qf[nt][kc][0], qf[nt][kc][1]);
        }
      }
      __syncwarp();  // every lane has read K
      if (i + 1 < n_valid) load(&k_map, bar_k, buf, i + 1);
      // keys past the query position (and past kv_len) are masked; log2 domain
      const int kpos0 = key0 + gi;
      auto scaled = [&](float x) { return kBlk ? fmaf(x, sl2, log2_vs) : x * sl2; };
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        const int ka = kpos0 + 16 * mt, kb2 = ka + 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          sacc[mt][nt][0] = ka <= qp[nt][0] ? scaled(sacc[mt][nt][0]) : -INFINITY;
          sacc[mt][nt][1] = ka <= qp[nt][1] ? scaled(sacc[mt][nt][1]) : -INFINITY;
          sacc[mt][nt][2] = kb2 <= qp[nt][0] ? scaled(sacc[mt][nt][2]) : -INFINITY;
          sacc[mt][nt][3] = kb2 <= qp[nt][1] ? scaled(sacc[mt][nt][3]) : -INFINITY;
        }
      }
      uint32_t pb[kMT][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float alpha[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(sacc[0][nt][c], sacc[0][nt][2 + c]);
#pragma unroll
          for (int mt = 1; mt < kMT; ++mt) mx = fmaxf(mx, fmaxf(sacc[mt][nt][c], sacc[mt][nt][2 + c]));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
          const float m_new = fmaxf(m[nt][c], mx);
          const float m_use = m_new == -INFINITY ? 0.f : m_new;
          alpha[c] = ex2_approx(m[nt][c] - m_use);
          m[nt][c] = m_new;
          float sum = 0.f;
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            sacc[mt][nt][c] = ex2_approx(sacc[mt][nt][c] - m_use);
            sacc[mt][nt][2 + c] = ex2_approx(sacc[mt][nt][2 + c] - m_use);
            sum += sacc[mt][nt][c] + sacc[mt][nt][2 + c];
          }
          l[nt][c] = l[nt][c] * alpha[c] + (kBlk ? sum * inv_vs : sum);
        }
#pragma unroll
        for (int md = 0; md < kMD; ++md) {
          oacc[md][nt][0] *= alpha[0];
          oacc[md][nt][2] *= alpha[0];
          oacc[md][nt][1] *= alpha[1];
          oacc[md][nt][3] *= alpha[1];
        }
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          pb[mt][nt][0] = movmatrix_t(pack_f16x2(sacc[mt][nt][0], sacc[mt][nt][1]));
          pb[mt][nt][1] = movmatrix_t(pack_f16x2(sacc[mt][nt][2], sacc[mt][nt][3]));
        }
      }
      if (!(ok = mbar_wait(bar_v, phase, err))) break;
      if (kBlk && key0 + kKeys - 1 > last) {  // the unit with the last query's own key
        for (int w = (last + 1 - key0) * (kD / 4) + lane; w < kKeys * (kD / 4); w += 32) sts32(vb + 4 * w, 0u);
        fence_async_shared();  // before the next load overwrites the buffer
        __syncwarp();
      }
      // O^T += V^T P^T over the unit's keys
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        const int r0 = 16 * mt + 2 * t4;
#pragma unroll
        for (int qg = 0; qg < kD / 32; ++qg) {
          const int col = 32 * qg + 4 * gi;
          const uint32_t w0 = lds32(vb + swz<kD>(r0, col)), w1 = lds32(vb + swz<kD>(r0 + 1, col));
          const uint32_t w2 = lds32(vb + swz<kD>(r0 + 8, col)), w3 = lds32(vb + swz<kD>(r0 + 9, col));
          const uint32_t x01 = prmt(w0, w1, 0x5140), x23 = prmt(w2, w3, 0x5140);
          const uint32_t y01 = prmt(w0, w1, 0x7362), y23 = prmt(w2, w3, 0x7362);
          const uint32_t a0 = e4m3x2_to_f16x2(x01), a1 = e4m3x2_to_f16x2(x01 >> 16);
          const uint32_t a2 = e4m3x2_to_f16x2(x23), a3 = e4m3x2_to_f16x2(x23 >> 16);
          const uint32_t b0 = e4m3x2_to_f16x2(y01), b1 = e4m3x2_to_f16x2(y01 >> 16);
          const uint32_t b2 = e4m3x2_to_f16x2(y23), b3 = e4m3x2_to_f16x2(y23 >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16(oacc[2 * qg][nt], a0, a1, a2, a3, pb[mt][nt][0], pb[mt][nt][1]);
            mma_f16(oacc[2 * qg + 1][nt], b0, b1, b2, b3, pb[mt][nt][0], pb[mt][nt][1]);
          }
        }
      }
      __syncwarp();  // every lane has read V
      if (i + 1 < n_valid) load(&v_map, bar_v, buf + kPartBytes, i + 1);
    }
  }

  // merge the warps' states: each warp's O goes to its own buffer ([head][128]
  // floats), (m, l) beside; then a thread takes four dims of one head
  float* sc = reinterpret_cast<float*>(buf);
  float2* ml = reinterpret_cast<float2*>(smem + L::kMlOff);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      l[nt][c] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][c], 4);
      l[nt][c] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][c], 8);
      l[nt][c] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][c], 16);
      const int h = 8 * nt + 2 * t4 + c;
      if (gi == 0) ml[warp * L::kHeads + h] = make_float2(ok ? m[nt][c] : -INFINITY, l[nt][c]);
#pragma unroll
      for (int md = 0; md < kMD; ++md) {
        const int d0 = 32 * (md >> 1) + 4 * gi + 2 * (md & 1);
        *reinterpret_cast<float2*>(sc + h * kD + d0) = make_float2(oacc[md][nt][c], oacc[md][nt][2 + c]);
      }
    }
  __syncthreads();
  // n states (m, l, O), `at(w)` the w-th one's (m, l) and `o(w)` its four dims
  auto merge = [&](int n, auto at, auto o) {
    float mm = -INFINITY;
    for (int w = 0; w < n; ++w) mm = fmaxf(mm, at(w).x);
    Merged r{mm, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int w = 0; w < n; ++w) {
      const float2 v = at(w);
      const float4 p = o(w);
      const float s = v.x == -INFINITY ? 0.f : ex2_approx(v.x - mm);
      r.l += v.y * s;
      r.o.x += p.x * s;
      r.o.y += p.y * s;
      r.o.z += p.z * s;
      r.o.w += p.w * s;
    }
    return r;
  };
  const float vs = kBlk ? 1.f : v_scale[kvh];
  auto write = [&](int h, int d4, const Merged& r) {
    const int64_t orow = static_cast<int64_t>(q_begin + row_of(h)) * hq + g * G + head_of(h);
    auto norm = [&](float x) { return r.l > 0.f ? x / r.l * vs : 0.f; };
    const __nv_bfloat162 a = __floats2bfloat162_rn(norm(r.o.x), norm(r.o.y));
    const __nv_bfloat162 b = __floats2bfloat162_rn(norm(r.o.z), norm(r.o.w));
    *reinterpret_cast<uint2*>(out + orow * kD + 4 * d4) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    if (d4 == 0 && lse != nullptr) lse[orow] = r.l > 0.f ? (r.m + log2f(r.l)) * 0.69314718055994531f : -INFINITY;
  };
  float4* cta_o = reinterpret_cast<float4*>(smem + L::kCtaOff);
  float2* cta_ml = ml + kWsWarps * L::kHeads;
  for (int e = threadIdx.x; e < H * (kD / 4); e += kWsThreads) {
    const int h = e / (kD / 4), d4 = e % (kD / 4);
    const Merged r = merge(
        kWsWarps, [&](int w) { return ml[w * L::kHeads + h]; },
        [&](int w) { return reinterpret_cast<const float4*>(smem + L::kBufOff + w * kBufBytes)[e]; });
    if (cs == 1) {
      write(h, d4, r);
    } else {
      cta_o[e] = r.o;
      if (d4 == 0) cta_ml[h] = make_float2(r.m, r.l);
    }
  }
  auto done = [&] {
    if (kFew && (chain & kFollows) && threadIdx.x == 0) pdl_wait();
  };
  if (cs == 1) return done();
  cluster_sync();  // the row's CTAs have written their states
  for (int e = rank * kWsThreads + threadIdx.x; e < H * (kD / 4); e += cs * kWsThreads) {
    const int h = e / (kD / 4);
    write(h, e % (kD / 4), merge(
        cs, [&](int w) { return ld_cluster_f2(smem_u32(cta_ml + h), w); },
        [&](int w) { return ld_cluster_f4(smem_u32(cta_o + e), w); }));
  }
  cluster_sync();  // nobody leaves while its state may be read
  done();
}

template <bool kBlk, int D, int NT, bool kFew = false>
cudaError_t launch_ws(const msa_plan_s* p, int n_tiles, const int2* part_list, int cs, cudaStream_t st, const CUtensorMap& km, const CUtensorMap& vm,
                      const void* q, const int32_t* kv_indices, const int32_t* idx, const float* k_scale,
                      const float* v_scale, void* out, float* lse) {
  auto kern = decode_ws_kernel<kBlk, D, NT, kFew>;
  const int smem = WsSmem<D, NT>::kBytes + 1024;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (cs > 8) cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  return launch_pdl_cluster(kern, dim3(n_tiles * p->hp * cs), cs, dim3(kWsThreads), smem, st, km, vm,
                            static_cast<const __nv_bfloat16*>(q), p->tiles_d, part_list, idx, kv_indices, p->num_pages, k_scale,
                            v_scale, static_cast<__nv_bfloat16*>(out), lse, p->hq, p->hp, p->hp / p->hkv, p->topk, cs,
                            1.4426950408889634f / sqrtf(static_cast<float>(D)), kFew && p->n_attn_units > 0 ? kFollows : 0,
                            p->err_d);
}

// CTAs a row: one for an SM at most, with a unit for every warp; clusters of
// 16 (beyond the portable 8) from four units a warp on.  Measured (us, block
// scales, d 128; the split over CTAs of decode.cu first, then cs = 1, 2, 4, ...):
//    8 rows, topk 16     18.2 | 11.8  9.4  7.6 [6.9]
//   32 rows, topk 16     19.4 | 11.9  9.5 [8.0] 8.8
//   64 rows, topk 16     21.2 | 13.6 [11.2] 11.2 18.2
//  128 rows, topk 16     27.0 | [16.5] 17.3 23.5
//  256 rows, topk 16     27.6 | [25.9] 32.6
//    8 rows, topk 64     40.6 | 35.7 21.4 13.8 [10.1] 10.8
//    1 row, topk 256      154 |  133  70  37  21 [14.2]
//    8 rows, topk 256    56.6 |  137  72  39  24 [21.3]
//   64 rows, topk 16, G 16  27.3 | 16.4 [12.9] 19.9
// Two CTAs of different clusters on one SM cost more than the second half of
// the row's parallelism brings.  Large clusters are not placed as densely as the
// SMs would allow: with one CTA an SM (two head tiles) 15 of 8 and 7 of 16 run at
// once (16 rows, G 16, topk 16: 8 CTAs a row 16.1 us, 4 9.4; 8 rows, topk 200: 16
// 32.1, 8 23.2).
int row_cluster(const msa_plan_s* p, int n_tiles, int ctas_per_sm) {
  const int rows = n_tiles * p->hp;
  auto fits = [&](int cs) { return cs < 8 || rows <= (cs == 8 ? 14 : 7) * ctas_per_sm; };
  int cs = 1;
  while (cs < 16 && rows * cs * 2 <= p->num_sms && 2 * cs * kWsWarps <= kParts * p->topk &&
         (cs < 8 || p->topk >= 128) && fits(2 * cs))
    cs *= 2;
  return cs;
}

}  // namespace

bool decode_ws_applies(const msa_plan_s* p) {
  if (p->kv_dtype == MSA_KV_FP8_E4M3_BLOCK) return true;
  return p->n_tiles * p->hp >= p->num_sms && p->hq / p->hp <= 8 && p->topk <= kMaxStaticTopk && p->d == 128;
}

msa_status launch_attn_decode_ws(const msa_plan_s* p, const void* q, const void* k_pages, const void* v_pages,
                                 const int32_t* kv_indices, const int32_t* idx, const float* k_scale,
                                 const float* v_scale, void* out, float* lse, cudaStream_t st) {
  const int2* part_list = p->n_row_parts > 0 ? reinterpret_cast<const int2*>(p->aux_d + p->row_parts_off) : nullptr;
  const int n_tiles = part_list ? p->n_row_parts : p->n_tiles;
  CUtensorMap km, vm;
  const uint64_t dims[2] = {static_cast<uint64_t>(p->d), static_cast<uint64_t>(p->num_pages) * p->hkv * 128};
  const uint64_t str[1] = {static_cast<uint64_t>(p->d)};
  const uint32_t box[2] = {static_cast<uint32_t>(p->d), static_cast<uint32_t>(kKeys)};
  if (!encode_tensor_map(&km, 2, k_pages, dims, str, box, 0, p->d) ||
      !encode_tensor_map(&vm, 2, v_pages, dims, str, box, 0, p->d))
    return set_error(MSA_ERR_CUDA, "msa_sparse_attn: tensor map encoding failed");
  const bool wide = (part_list ? p->row_part_heads : p->hq / p->hp) > 8;
  const auto launch =
      p->kv_dtype != MSA_KV_FP8_E4M3_BLOCK ? launch_ws<false, 128, 1>
      : part_list ? (p->d == 128 ? (wide ? launch_ws<true, 128, 2, true> : launch_ws<true, 128, 1, true>)
                                 : (wide ? launch_ws<true, 64, 2, true> : launch_ws<true, 64, 1, true>))
                  : (p->d == 128 ? (wide ? launch_ws<true, 128, 2> : launch_ws<true, 128, 1>)
                                 : (wide ? launch_ws<true, 64, 2> : launch_ws<true, 64, 1>));
  const int cs = p->kv_dtype == MSA_KV_FP8_E4M3_BLOCK ? row_cluster(p, n_tiles, wide ? 1 : 2) : 1;
  return cuda_check(launch(p, n_tiles, part_list, cs, st, km, vm, q, kv_indices, idx, k_scale, v_scale, out, lse),
                    "msa_sparse_attn: decode launch");
}

}  // namespace msa
