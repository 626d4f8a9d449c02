// Rotary positions: the rotation of query and key heads by their positions,
// and its transpose for the gradients.
//
//   pair (a, b) of a head, angle t = 2 pi turns_i position:
//   a' = m (a cos t - b sin t),  b' = m (b cos t + a sin t)
// Dims from rotary_dim on are copied.  The inverse rotates by -t with the
// same factor m: it is the transpose of the forward map, so it takes the
// gradient of the rotated heads to the gradient of the heads.
//
// Bound by HBM: every element is read and written once and costs three
// multiply-adds.  A CTA takes the rows' memory in order (a row is its heads, one
// after the other), with the cos and sin of its rows in shared memory, computed
// once for all heads; a thread rotates 16 values at a time (both members of
// eight pairs) and has the loads of kBatch such chunks in flight before the
// first store, which the compiler cannot move them across.
// bf16, 32768 rows x 32 heads of 128 (0.54 GB): 85 us, 6.3 TB/s (a copy of as
// much takes 82); fp32, 65536 x 32 (2.1 GB): 310 us, 6.9 TB/s.
#include <math.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "ptx.cuh"
#include "rope.cuh"

namespace msa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeSmem = 16384;  // bytes of angles a CTA at most

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeTable tab, const T* x, int64_t x_stride, const int32_t* __restrict__ pos,
                int64_t n_rows, int32_t heads, int32_t d, bool inverse, int32_t cta_rows, int32_t cta_heads, T* out,
                int64_t out_stride) {
  pdl_wait();
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;
  extern __shared__ float4 angles[];  // [row][4][rot / 16]: cos, cos, sin, sin of pairs 2 j and 2 j + 1 of a chunk
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * cta_rows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(cta_rows), n_rows - row0));
  const int h0 = blockIdx.y * cta_heads, nh = min(cta_heads, heads - h0);
  // thread: chunk c of the (row, head) items j, j + step, ...
  const int chunks = d / 16, step = kRopeThreads / chunks, turning = tab.rot / 16;
  const int c = threadIdx.x % chunks, j = threadIdx.x / chunks;
  const RopeChunk ch = rope_chunk(tab, c);
  const int n = j < step && (ch.rotated || x != out) ? rows * nh : 0;  // in place: the unrotated stay
  const T* xr = x + row0 * x_stride + h0 * d;
  T* orow = out + row0 * out_stride + h0 * d;
  const int step_r = step / nh, step_h = step % nh;
  int r = j / nh, h = j % nh;  // of item i
  bool first = true;
  for (int i = j; i < n || first; i += kBatch * step) {
    Raw16<T> raw[kBatch];
    int rr[kBatch], hh[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      rr[b] = r, hh[b] = h;
      if (i + b * step < n) raw[b].load(xr + r * x_stride + h * d + ch.lo, xr + r * x_stride + h * d + ch.hi);
      r += step_r, h += step_h;
      if (h >= nh) h -= nh, ++r;
    }
    if (first) {  // while the first loads are on their way
      for (int a = threadIdx.x; a < rows * turning; a += kRopeThreads) {
        const int ar = a / turning, ac = a % turning;
        float cs[8], sn[8];
        rope_angles(tab, ac, pos[row0 + ar], inverse, cs, sn);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          angles[(ar * 4 + k) * turning + ac] = make_float4(cs[2 * k], cs[2 * k + 1], sn[2 * k], sn[2 * k + 1]);
      }
      __syncthreads();
      first = false;
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (i + b * step >= n) break;
      float v[16];
      raw[b].unpack(v);
      if (ch.rotated) {
#pragma unroll
        for (int k = 0; k < 4; ++k) rope_rotate2(INTERLEAVED, k, angles[(rr[b] * 4 + k) * turning + c], v);
      }
      T* o = orow + rr[b] * out_stride + hh[b] * d;
      store8(o + ch.lo, v);
      store8(o + ch.hi, v + 8);
    }
  }
}

template <typename T>
msa_status launch_rope(const RopeTable& tab, const void* x, int64_t xs, const int32_t* pos, int64_t n_rows,
                       int32_t heads, int32_t d, bool inverse, void* out, int64_t os, int num_sms, cudaStream_t st) {
  // a CTA's items: kItems chunks a thread (512 bytes read), of whole rows where
  // a row has no more; fewer where that leaves SMs without a CTA.  bf16, 32768
  // rows x 32 heads (shorter angle polynomials): 4 items 88 us, 8 83, 16 81, 32 86; fp32, 65536 x 32: 4 304,
  // 8 309, 16 316, 32 325.  4096 x 8: a CTA an SM 5.2 us, 4 an SM 6.8
  const int64_t chunks = d / 16, total = n_rows * heads * chunks;
  constexpr int kItems = 32 / sizeof(T);
  const int64_t per = std::clamp<int64_t>(total / num_sms, kRopeThreads, kItems * kRopeThreads) / chunks;
  const int cta_heads = static_cast<int>(std::min<int64_t>(heads, per));
  const int cta_rows = static_cast<int>(
      std::clamp<int64_t>(per / heads, 1, std::min<int64_t>(n_rows, kRopeSmem / (tab.rot * 4))));
  const int64_t gx = (n_rows + cta_rows - 1) / cta_rows;
  if (gx > 0x7FFFFFFF) return set_error(MSA_ERR_INVALID_ARG, "msa_rope_apply: too many rows");
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>((heads + cta_heads - 1) / cta_heads));
  const auto kern = tab.interleaved ? rope_kernel<T, true> : rope_kernel<T, false>;
  return cuda_check(launch_pdl(kern, grid, dim3(kRopeThreads), size_t(cta_rows) * tab.rot * 4, st, tab,
                               static_cast<const T*>(x), xs, pos, n_rows, heads, d, inverse, cta_rows, cta_heads,
                               static_cast<T*>(out), os),
                    "msa_rope_apply: launch");
}

// Double-double numbers hi + lo (Dekker 1971, Knuth's two-sum): the table holds
// 64 bits of a turn, and a position of 2^31 leaves the phase an error of 2^31
// times the table's.
struct DD {
  double hi, lo;
};
DD two_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
DD operator+(DD a, DD b) {
  const DD s = two_sum(a.hi, b.hi);
  return two_sum(s.hi, s.lo + (a.lo + b.lo));
}
DD operator*(DD a, DD b) {
  const double p = a.hi * b.hi;
  return two_sum(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
DD operator-(DD a) { return {-a.hi, -a.lo}; }
DD operator/(DD a, DD b) {
  const double q = a.hi / b.hi;
  const DD r = a + -(b * DD{q, 0.0});
  return two_sum(q, r.hi / b.hi);
}
// 2^k e^r with |r| <= ln 2 / 2, e^r as the 2^9th power of a Taylor sum; 1 is kept
// apart until the end, since the squarings would multiply its rounding
DD dd_exp(DD x) {
  const DD ln2{0x1.62e42fefa39efp-1, 0x1.abc9e3b39803fp-56};
  const double k = std::nearbyint(x.hi / ln2.hi);
  DD r = x + -(ln2 * DD{k, 0.0});
  r = {std::ldexp(r.hi, -9), std::ldexp(r.lo, -9)};
  DD e{0.0, 0.0};  // e^r - 1, |r| < 2^-10: the first term left out is below 2^-120
  for (int n = 10; n >= 1; --n) e = (DD{1.0, 0.0} + e) * r / DD{static_cast<double>(n), 0.0};
  for (int i = 0; i < 9; ++i) e = DD{2 * e.hi, 2 * e.lo} + e * e;
  e = DD{1.0, 0.0} + e;
  return {std::ldexp(e.hi, static_cast<int>(k)), std::ldexp(e.lo, static_cast<int>(k))};
}
// one Newton step on e^y = x
DD dd_log(double x) {
  const DD y{std::log(x), 0.0};
  return y + (DD{x, 0.0} * dd_exp(-y) + DD{-1.0, 0.0});
}
// x in [0, 1/2) in units of 2^-64, to the nearest
uint64_t fraction64(DD x) {
  const double a = std::ldexp(x.hi, 64), whole = std::floor(a);
  return static_cast<uint64_t>(whole) + static_cast<uint64_t>(std::llrint((a - whole) + std::ldexp(x.lo, 64)));
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

msa_status msa_rope_create(int32_t rotary_dim, msa_rope_layout layout, double base, msa_rope_scaling scaling,
                           double factor, int32_t original_len, double beta_fast, double beta_slow, msa_rope_t* out) {
  const char* fn = "msa_rope_create";
  if (!out) return set_error(MSA_ERR_INVALID_ARG, "%s: out is NULL", fn);
  *out = nullptr;
  if (rotary_dim < 16 || rotary_dim % 16 != 0 || rotary_dim > 2 * kMaxRopePairs)
    return set_error(MSA_ERR_UNSUPPORTED, "%s: rotary_dim must be a multiple of 16 in [16, %d]", fn,
                     2 * kMaxRopePairs);
  if (layout != MSA_ROPE_HALF && layout != MSA_ROPE_INTERLEAVED)
    return set_error(MSA_ERR_INVALID_ARG, "%s: unknown layout", fn);
  if (!(base > 1.0) || !isfinite(base)) return set_error(MSA_ERR_INVALID_ARG, "%s: base must be above 1", fn);
  if (scaling < MSA_ROPE_NONE || scaling > MSA_ROPE_YARN)
    return set_error(MSA_ERR_INVALID_ARG, "%s: unknown scaling", fn);
  if (scaling != MSA_ROPE_NONE && (!(factor >= 1.0) || !isfinite(factor)))
    return set_error(MSA_ERR_INVALID_ARG, "%s: factor must be at least 1", fn);
  if (scaling == MSA_ROPE_YARN &&
      (original_len < 1 || !(beta_fast >= beta_slow) || !(beta_slow > 0.0) || !isfinite(beta_fast)))
    return set_error(MSA_ERR_INVALID_ARG, "%s: YaRN needs original_len >= 1 and beta_fast >= beta_slow > 0", fn);
  auto* r = new (std::nothrow) msa_rope_s();
  if (!r) return set_error(MSA_ERR_NO_MEMORY, "%s: out of host memory", fn);
  const double two_pi = 6.283185307179586476925;
  const int pairs = rotary_dim / 2;
  DD log_base = dd_log(base);
  if (scaling == MSA_ROPE_NTK)
    log_base = log_base + dd_log(factor) * (DD{double(rotary_dim), 0.0} / DD{rotary_dim - 2.0, 0.0});
  // YaRN: pairs that turn more than beta_fast times over the original length
  // keep their frequency, those below beta_slow are interpolated, a linear
  // ramp over the pair index joins them
  double lo = 0.0, width = 1.0;
  if (scaling == MSA_ROPE_YARN) {
    auto dim = [&](double beta) { return rotary_dim * log(original_len / (two_pi * beta)) / (2.0 * log(base)); };
    lo = std::max(floor(dim(beta_fast)), 0.0);
    width = std::max(std::min(ceil(dim(beta_slow)), rotary_dim - 1.0) - lo, 1e-3);
  }
  for (int i = 0; i < pairs; ++i) {
    const DD one{1.0, 0.0}, inv_two_pi{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57}, f{factor, 0.0};
    DD turns = dd_exp(log_base * (DD{-2.0 * i, 0.0} / DD{double(rotary_dim), 0.0})) * inv_two_pi;
    if (scaling == MSA_ROPE_LINEAR) turns = turns / f;
    if (scaling == MSA_ROPE_YARN) {
      DD ramp = DD{i - lo, 0.0} / DD{width, 0.0};
      if (ramp.hi <= 0.0) ramp = {0.0, 0.0};
      if (ramp.hi >= 1.0) ramp = one;
      turns = turns * (one + -ramp) + turns / f * ramp;
    }
    r->table.turns[i] = fraction64(turns);  // turns <= 1 / (2 pi)
  }
  const double m = scaling == MSA_ROPE_YARN && factor > 1.0 ? 0.1 * log(factor) + 1.0 : 1.0;
  r->table.mscale = static_cast<float>(m);
  r->table.mscale_lo = static_cast<float>(m - static_cast<double>(r->table.mscale));
  r->table.rot = rotary_dim;
  r->table.interleaved = layout == MSA_ROPE_INTERLEAVED;
  *out = r;
  return MSA_OK;
}

void msa_rope_destroy(msa_rope_t rope) { delete rope; }

msa_status msa_rope_apply(msa_rope_t rope, const void* x, int64_t x_row_stride, const int32_t* positions,
                          int64_t n_rows, int32_t heads, int32_t head_dim, msa_dtype dtype, int32_t inverse,
                          void* out, int64_t out_row_stride, msa_stream_t stream) {
  const char* fn = "msa_rope_apply";
  if (!rope) return set_error(MSA_ERR_INVALID_ARG, "%s: NULL argument", fn);
  if (n_rows < 0 || heads < 1 || heads > 65535 || head_dim < 16)
    return set_error(MSA_ERR_INVALID_ARG, "%s: sizes out of range", fn);
  if (dtype != MSA_BF16 && dtype != MSA_F32) return set_error(MSA_ERR_INVALID_ARG, "%s: unknown dtype", fn);
  if (head_dim % 16 != 0 || head_dim > 256)
    return set_error(MSA_ERR_UNSUPPORTED, "%s: head_dim must be a multiple of 16 up to 256", fn);
  if (rope->table.rot > head_dim)
    return set_error(MSA_ERR_INVALID_ARG, "%s: rotary_dim %d above head_dim %d", fn, rope->table.rot, head_dim);
  if (n_rows == 0) return MSA_OK;
  if (!x || !positions || !out) return set_error(MSA_ERR_INVALID_ARG, "%s: NULL argument", fn);
  const int64_t es = dtype == MSA_BF16 ? 2 : 4, width = int64_t(heads) * head_dim;
  if (x_row_stride < width || out_row_stride < width || x_row_stride > (int64_t(1) << 40) ||
      out_row_stride > (int64_t(1) << 40))
    return set_error(MSA_ERR_INVALID_ARG, "%s: row strides must be at least heads * head_dim", fn);
  if (!aligned16(x) || !aligned16(out) || x_row_stride * es % 16 != 0 || out_row_stride * es % 16 != 0)
    return set_error(MSA_ERR_INVALID_ARG, "%s: rows must start on 16-byte boundaries", fn);
  if (!rows_disjoint_or_same(x, x_row_stride * es, out, out_row_stride * es, n_rows, width * es))
    return set_error(MSA_ERR_INVALID_ARG, "%s: out overlaps x without being x itself", fn);
  int dev = 0, sms = 0;
  msa_status s = cuda_check(cudaGetDevice(&dev), "msa_rope_apply: cudaGetDevice");
  if (s == MSA_OK)
    s = cuda_check(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "msa_rope_apply: SM count");
  if (s != MSA_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == MSA_BF16 ? launch_rope<__nv_bfloat16>(rope->table, x, x_row_stride, positions, n_rows, heads,
                                                        head_dim, inverse != 0, out, out_row_stride, sms, st)
                           : launch_rope<float>(rope->table, x, x_row_stride, positions, n_rows, heads, head_dim,
                                                inverse != 0, out, out_row_stride, sms, st);
}

}  // extern "C"
