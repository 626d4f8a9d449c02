"""ctypes binding of libmsa (include/msa.h): argument marshalling only.

Every step of the hot path runs in libmsa's CUDA kernels.  Torch tensors
supply device memory and the current stream; this module checks dtypes,
shapes and contiguity, passes data_ptr()s, and raises MsaError on any
non-OK status.  Importing it fails loudly when libmsa.so is missing.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmsa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libmsa.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_u32 = ctypes.c_uint32
_f32 = ctypes.c_float
_f64 = ctypes.c_double

STATUS = {0: "MSA_OK", 1: "MSA_ERR_INVALID_ARG", 2: "MSA_ERR_UNSUPPORTED", 3: "MSA_ERR_CUDA",
          4: "MSA_ERR_NO_MEMORY", 5: "MSA_ERR_TIMEOUT", 6: "MSA_ERR_DEVICE_CHECK",
          7: "MSA_ERR_NONFINITE"}
KV_BF16, KV_FP8_E4M3, KV_FP8_E4M3_BLOCK = 0, 1, 2
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

# Every symbol include/msa.h declares, with its ctypes signature.
SIGNATURES = {
    "msa_plan": (_i32, [_p, _p, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i64, _i32, _u32, _p, _p]),
    "msa_plan_destroy": (None, [_p]),
    "msa_plan_num_tiles": (_i32, [_p]),
    "msa_plan_max_blocks": (_i32, [_p]),
    "msa_plan_total_q": (_i64, [_p]),
    "msa_plan_num_valid_pages": (_p, [_p]),
    "msa_proxy_maxscore": (_i32, [_p, _p, _p, _p, _p, _p]),
    "msa_proxy_maxscore_fp8": (_i32, [_p, _p, _p, _p, _p, _p, _p]),
    "msa_proxy_maxscore_nvfp4": (_i32, [_p, _p, _p, _p, _p, _p, _p, _p]),
    "msa_proxy_topk": (_i32, [_p, _p, _p, _p, _p, _p, _p]),
    "msa_topk_select": (_i32, [_p, _i32, _i32, _i32, _i32, _p, _p, _p]),
    "msa_sparse_attn": (_i32, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p]),
    "msa_sparse_attn_bwd": (_i32, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _f32, _p, _p, _p, _p, _p, _p]),
    "msa_sparse_decode_noalloc": (_i32, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _i32, _i32, _i32, _i32, _i32, _i64,
                                         _p, _p, _p, _p]),
    "msa_rope_create": (_i32, [_i32, _i32, _f64, _i32, _f64, _i32, _f64, _f64, _p]),
    "msa_rope_destroy": (None, [_p]),
    "msa_rope_apply": (_i32, [_p, _p, _i64, _p, _i64, _i32, _i32, _i32, _i32, _p, _i64, _p]),
    "msa_kv_append": (_i32, [_p, _p, _p, _p, _i64, _p, _i64, _p, _p, _p, _p, _p, _p]),
    "msa_pk_append": (_i32, [_p, _p, _p, _p, _i64, _p, _p, _p, _p, _p, _p, _p, _p]),
    "msa_append_bwd": (_i32, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p]),
    "msa_tree_attn": (_i32, [_p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _p]),
    "msa_latent_append": (_i32, [_p, _p, _p, _p, _i64, _p, _i64, _p, _i32, _i32, _p, _p]),
    "msa_latent_attn": (_i32, [_p, _p, _p, _p, _p, _p, _i32, _i32, _f32, _p, _p, _p]),
    "msa_latent_expand": (_i32, [_p, _p, _p, _p, _p, _i32, _i32, _p, _p, _p]),
    "msa_check_errors": (_i32, [_p, _p]),
    "msa_selftest_wait_timeout": (_i32, [_p]),
    "msa_test_fail_plan_allocs": (None, [_i32]),
    "msa_last_error": (ctypes.c_char_p, []),
    "msa_version": (ctypes.c_char_p, []),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class MsaError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = _lib.msa_last_error().decode()
        super().__init__("%s: %s (%s)" % (where, STATUS.get(status, status), msg))


def _check(status, where):
    if status != 0:
        raise MsaError(status, where)


_current_device = torch._C._cuda_getDevice
# Two private parts of torch that save host time; one without them does without.
_guards = getattr(getattr(torch._C, "_dynamo", None), "guards", None)
# (shape, strides, dtype) on the current device, without the dispatcher: two outputs by
# torch.empty take 3.5 us more of a call that takes 10
_new = getattr(_guards, "_empty_strided_cuda", None) or (
    lambda shape, strides, dtype: torch.empty(shape, dtype=dtype, device="cuda"))
# type, dtype, device, sizes and strides of several tensors against those it was made of
_Alike = getattr(_guards, "TensorGuards", None)

# The checks and conversions below run several times a call, and a decode step's
# kernels are as short as they are: what passes is decided in one expression.

def _stream(stream=None):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(_current_device())
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, dtype, shape, name):
    if t.dtype is dtype and t.shape == shape and t.get_device() == _current_device() and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError("%s: dtype %s, want %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s: shape %s, want %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_cuda or not t.is_contiguous() or t.get_device() != _current_device():
        raise ValueError("%s: must be a contiguous CUDA tensor on the current device" % name)


def _need_all(tensors, needs, optional=False):
    """_need of several tensors, None passed over where `optional`; needs: their
    (dtype, shape, name)."""
    dev = _current_device()
    for t, need in zip(tensors, needs):
        if t is None and optional:
            continue
        dtype, shape, _ = need
        if not (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
            _need(t, *need)


def _rows(t, dtype, shape, name):
    """_need for rows at a stride: the heads of a row dense, the rows anywhere
    apart (a slice of a fused projection).  Returns that stride."""
    n, heads, d = shape
    if t.dtype is dtype and t.shape == shape and t.get_device() == _current_device():
        row, head, one = t.stride()
        if one == 1 and (head == d or heads == 1):
            return row if n > 1 else heads * d
    if t.dtype != dtype:
        raise TypeError("%s: dtype %s, want %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s: shape %s, want %s" % (name, tuple(t.shape), tuple(shape)))
    if t.numel() == 0 and t.is_cuda:
        return heads * d
    raise ValueError("%s: must be a CUDA tensor with dense rows on the current device" % name)


def version():
    return _lib.msa_version().decode()


def selftest_wait_timeout(stream=None):
    """Runs the device-side failure path once (msa_selftest_wait_timeout): a
    kernel whose bounded wait cannot complete gives up after its limit.
    Raises MsaError with status MSA_ERR_TIMEOUT, as a timed-out kernel would
    through check_errors."""
    _check(_lib.msa_selftest_wait_timeout(_stream(stream)), "msa_selftest_wait_timeout")


def inject_plan_alloc_failures(count):
    """Failure injection (msa_test_fail_plan_allocs): the next `count` plan
    creations fail at their device allocation with MSA_ERR_NO_MEMORY."""
    _lib.msa_test_fail_plan_allocs(int(count))


def topk_select(max_score, topk, num_valid_pages, out=None, stream=None):
    """kv_block_indexes [n_tiles, heads, topk] int32 from max_score [n_tiles,
    heads, max_blocks] fp32 (msa_topk_select)."""
    n, h, nb = max_score.shape
    _need(max_score, torch.float32, (n, h, nb), "max_score")
    _need(num_valid_pages, torch.int32, (n,), "num_valid_pages")
    if out is None:
        out = torch.empty((n, h, topk), dtype=torch.int32, device=max_score.device)
    _need(out, torch.int32, (n, h, topk), "kv_block_indexes")
    _check(_lib.msa_topk_select(_ptr(max_score), n, h, nb, topk, _ptr(num_valid_pages), _ptr(out),
                                _stream(stream)), "msa_topk_select")
    return out


def sparse_decode_noalloc(q, k_pages, v_pages, kv_lens, kv_indptr, kv_indices, kv_block_indexes, k_scale,
                          v_scale, out=None, lse=None, err_word=None, stream=None):
    """FP8 paged decode without a plan and without any device allocation by
    the library (msa_sparse_decode_noalloc): the batch comes as device
    int32 kv_lens [B] and kv_indptr [B+1]; scratch is libmsa's static
    array.  Outputs may be passed in (out bf16 [B, Hq, 128], lse fp32
    [B, Hq], err_word uint32/int32 [1])."""
    b, hq, d = q.shape
    hkv = k_pages.shape[1]
    topk = kv_block_indexes.shape[2]
    _need(q, torch.bfloat16, (b, hq, d), "q")
    _need(k_pages, torch.float8_e4m3fn, tuple(k_pages.shape), "k_pages")
    _need(v_pages, torch.float8_e4m3fn, tuple(k_pages.shape), "v_pages")
    _need(kv_lens, torch.int32, (b,), "kv_lens")
    _need(kv_indptr, torch.int32, (b + 1,), "kv_indptr")
    _need(kv_indices, torch.int32, (kv_indices.numel(),), "kv_indices")
    _need(kv_block_indexes, torch.int32, (b, hkv, topk), "kv_block_indexes")
    _need(k_scale, torch.float32, (hkv,), "k_scale")
    _need(v_scale, torch.float32, (hkv,), "v_scale")
    if out is None:
        out = torch.empty_like(q)
    _need(out, torch.bfloat16, (b, hq, d), "out")
    if lse is not None:
        _need(lse, torch.float32, (b, hq), "lse")
    if err_word is not None:
        if err_word.dtype not in (torch.int32, torch.uint32) or err_word.numel() != 1:
            raise TypeError("err_word: want one 4-byte integer, got %s %s" % (err_word.dtype, tuple(err_word.shape)))
        if not err_word.is_cuda:
            raise ValueError("err_word: must be a CUDA tensor")
    _check(_lib.msa_sparse_decode_noalloc(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(kv_lens), _ptr(kv_indptr),
                                          _ptr(kv_indices), _ptr(kv_block_indexes), _ptr(k_scale), _ptr(v_scale),
                                          b, hq, hkv, d, topk, k_pages.shape[0], _ptr(out), _ptr(lse),
                                          _ptr(err_word), _stream(stream)), "msa_sparse_decode_noalloc")
    return out, lse


class Rope:
    """Rotary frequencies (msa_rope_create): rotary_dim dims of a head turn in
    pairs, (i, i + rotary_dim/2) for "half" and (2i, 2i + 1) for
    "interleaved"; scaling "none", "linear", "ntk" or "yarn" by factor."""

    def __init__(self, rotary_dim, layout="half", base=10000.0, scaling="none", factor=1.0, original_len=0,
                 beta_fast=32.0, beta_slow=1.0):
        self.rotary_dim = int(rotary_dim)
        h = ctypes.c_void_p()
        _check(_lib.msa_rope_create(self.rotary_dim, ROPE_LAYOUTS[layout], float(base), ROPE_SCALINGS[scaling],
                                    float(factor), int(original_len), float(beta_fast), float(beta_slow),
                                    ctypes.byref(h)), "msa_rope_create")
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            _lib.msa_rope_destroy(h)
            self._h = None

    def apply(self, x, positions, out=None, inverse=False, stream=None):
        """x [rows, heads, head_dim] (bf16 or fp32, rows at a stride) rotated by
        int32 positions [rows], or back with inverse=True, which is the
        gradient (msa_rope_apply).  out may be x."""
        dtype, shape = x.dtype, x.shape
        if dtype is not torch.bfloat16 and dtype is not torch.float32:
            raise TypeError("x: dtype %s, want bfloat16 or float32" % dtype)
        n, heads, d = shape
        x_stride = _rows(x, dtype, shape, "x")
        _need(positions, torch.int32, (n,), "positions")
        if out is None:
            out, out_stride = torch.empty(shape, dtype=dtype, device=x.device), heads * d
        else:
            out_stride = _rows(out, dtype, shape, "out")
        _check(_lib.msa_rope_apply(self._h, x.data_ptr(), x_stride, positions.data_ptr(), n, heads, d,
                                   dtype is torch.float32, inverse, out.data_ptr(), out_stride, _stream(stream)),
               "msa_rope_apply")
        return out


class _PlanHandle(ctypes.c_void_p):
    """A plan of libmsa, destroyed with the last that refers to it: the Plan, or a
    view of its device tables."""

    def __del__(self):
        if self.value:
            _lib.msa_plan_destroy(self)
            self.value = None


class Plan:
    """A validated batch shape with its device tables (msa_plan)."""

    def __init__(self, qo_lens, kv_lens, num_qo_heads, num_kv_heads, num_proxy_heads, head_dim, proxy_head_dim,
                 topk, num_pages, kv_dtype="bf16", page_size=128, stream=None):
        self.qo_lens = [int(x) for x in qo_lens]
        self.kv_lens = [int(x) for x in kv_lens]
        b = len(self.qo_lens)
        qa = (ctypes.c_int32 * b)(*self.qo_lens)
        ka = (ctypes.c_int32 * b)(*self.kv_lens)
        self.hq, self.hkv, self.hp, self.d, self.dp, self.topk = (num_qo_heads, num_kv_heads, num_proxy_heads,
                                                                  head_dim, proxy_head_dim, topk)
        self.num_pages = int(num_pages)
        self.kv_dtype = kv_dtype
        code = {"bf16": KV_BF16, "e4m3": KV_FP8_E4M3, "e4m3_block": KV_FP8_E4M3_BLOCK}[kv_dtype]
        h = _PlanHandle()
        _check(_lib.msa_plan(qa, ka, b, num_qo_heads, num_kv_heads, num_proxy_heads, head_dim, proxy_head_dim,
                             page_size, topk, self.num_pages, code, 0, _stream(stream), ctypes.byref(h)),
               "msa_plan")
        self._h = h
        self.n_tiles = _lib.msa_plan_num_tiles(h)
        self.max_blocks = _lib.msa_plan_max_blocks(h)
        self.total_q = _lib.msa_plan_total_q(h)
        self.n_page_entries = sum((k + 127) // 128 for k in self.kv_lens)
        # an int32 view of the plan's device num_valid_pages table
        nvp_ptr = _lib.msa_plan_num_valid_pages(h)
        self._nvp_raw = nvp_ptr
        self.num_valid_pages = _device_view_int32(nvp_ptr, self.n_tiles, torch.cuda.current_device(), h)
        self.num_valid_pages_host = None
        # what the calls around a step check of their tensors, made once
        kvt = torch.bfloat16 if kv_dtype == "bf16" else torch.float8_e4m3fn
        pool = (self.num_pages, self.hkv, 128, self.d)
        self._rows_shape = (self.total_q, self.hkv, self.d)
        self._q_shape, self._lse_shape = (self.total_q, self.hq, self.d), (self.total_q, self.hq)
        self._cache_needs = ((torch.int32, (self.n_page_entries,), "kv_indices"), (kvt, pool, "k_pages"),
                             (kvt, pool, "v_pages"))
        if kv_dtype != "bf16":
            shape = (self.hkv,) if kv_dtype == "e4m3" else (self.num_pages, self.hkv)
            self._cache_needs += ((torch.float32, shape, "k_scale"), (torch.float32, shape, "v_scale"))
        pos, ppool = (torch.int32, (self.total_q,), "positions"), (self.num_pages, 1, 128)
        self._pk_needs = ((torch.bfloat16, ppool + (self.dp,), "pk_pages"),
                          (torch.float8_e4m3fn, ppool + (self.dp,), "pk_pages_e4m3"), (torch.float32, (1,), "pk_scale"),
                          (torch.uint8, ppool + (self.dp // 2,), "pk_codes"),
                          (torch.float8_e4m3fn, ppool + (self.dp // 16,), "pk_block_scales"),
                          (torch.float32, (1,), "pk_global_scale"), pos, self._cache_needs[0])
        self._pk_shape = (self.total_q, 1, self.dp)
        self._grad_needs = ((torch.float32, pool, "dk_pages"), (torch.float32, pool, "dv_pages"),
                            (torch.float32, ppool + (self.dp,), "dpk_pages"), pos, self._cache_needs[0])
        self._attn_needs = self._cache_needs + ((torch.bfloat16, self._q_shape, "q"), (
            torch.int32, (self.n_tiles, self.hp, self.topk), "kv_block_indexes"))
        self._tree_needs = self._attn_needs + ((torch.int32, (self.total_q, 4), "tree_mask"),)
        self._table_needs = (self._cache_needs[0],) + self._tree_needs[-2:]
        self._alike = {}

    # -- the cache
    def kv_append(self, k, v, k_pages, v_pages, kv_indices, k_scale=None, v_scale=None, rope=None, positions=None,
                  stream=None):
        """The batch's new K and V rows [total_q, Hkv, d] bf16 into the cache
        (msa_kv_append), K rotated by `rope` at int32 positions [total_q], or at
        its key positions; quantised by the plan's kv_dtype."""
        k_stride = _rows(k, torch.bfloat16, self._rows_shape, "k")
        v_stride = _rows(v, torch.bfloat16, self._rows_shape, "v")
        _need_all((kv_indices, k_pages, v_pages) if self.kv_dtype == "bf16" else
                  (kv_indices, k_pages, v_pages, k_scale, v_scale), self._cache_needs)
        if positions is not None:
            _need(positions, torch.int32, (self.total_q,), "positions")
        _check(_lib.msa_kv_append(self._h, rope and rope._h, _ptr(positions), k.data_ptr(), k_stride, v.data_ptr(),
                                  v_stride, kv_indices.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                  _ptr(k_scale), _ptr(v_scale), _stream(stream)), "msa_kv_append")

    def pk_append(self, pk, kv_indices, pk_pages=None, pk_pages_e4m3=None, pk_scale=None, pk_codes=None,
                  pk_block_scales=None, pk_global_scale=None, rope=None, positions=None, stream=None):
        """The batch's new proxy K rows [total_q, 1, dp] bf16 into the pools given
        (msa_pk_append): bf16, e4m3 with pk_scale, NVFP4 with its scales."""
        pk_stride = _rows(pk, torch.bfloat16, self._pk_shape, "pk")
        _need_all((pk_pages, pk_pages_e4m3, pk_scale, pk_codes, pk_block_scales, pk_global_scale, positions, kv_indices),
                  self._pk_needs, optional=True)
        _check(_lib.msa_pk_append(self._h, rope and rope._h, _ptr(positions), pk.data_ptr(), pk_stride,
                                  kv_indices.data_ptr(), _ptr(pk_pages), _ptr(pk_pages_e4m3), _ptr(pk_scale),
                                  _ptr(pk_codes), _ptr(pk_block_scales), _ptr(pk_global_scale), _stream(stream)),
               "msa_pk_append")

    def append_bwd(self, kv_indices, dk_pages=None, dv_pages=None, dpk_pages=None, k_rope=None, pk_rope=None,
                   positions=None, stream=None):
        """Gradients of the appended rows from the gradient pages of
        sparse_attn_bwd (msa_append_bwd): (dk, dv [total_q, Hkv, d], dpk
        [total_q, 1, dp]) fp32, None where no pages are given."""
        _need_all((dk_pages, dv_pages, dpk_pages, positions, kv_indices), self._grad_needs, optional=True)
        dev = kv_indices.device
        dk, dv, dpk = (None if pages is None else torch.empty(shape, dtype=torch.float32, device=dev)
                       for pages, shape in ((dk_pages, self._rows_shape), (dv_pages, self._rows_shape),
                                            (dpk_pages, self._pk_shape)))
        _check(_lib.msa_append_bwd(self._h, k_rope and k_rope._h, pk_rope and pk_rope._h, _ptr(positions),
                                   kv_indices.data_ptr(), _ptr(dk_pages), _ptr(dv_pages), _ptr(dpk_pages), _ptr(dk),
                                   _ptr(dv), _ptr(dpk), _stream(stream)), "msa_append_bwd")
        return dk, dv, dpk

    def latent_append(self, latent, key, latent_pages, kv_indices, rope=None, positions=None, stream=None):
        """The batch's new rows of a latent cache (msa_latent_append): latent
        [total_q, 1, latent_dim] and key [total_q, 1, rope_dim] bf16, at strides,
        into latent_pages [P, 1, 128, latent_dim + rope_dim]; key rotated by
        `rope` at int32 positions [total_q], or at its key positions."""
        n, width = latent.shape[-1], key.shape[-1]
        tensors = (latent, key, latent_pages, kv_indices)
        if positions is not None:
            tensors += (positions,)
        known = strides = self._passed("latent_append", tensors)
        if known is None:
            strides = (_rows(latent, torch.bfloat16, (self.total_q, 1, n), "latent"),
                       _rows(key, torch.bfloat16, (self.total_q, 1, width), "key"))
            _need_all(tensors[2:], ((torch.bfloat16, (self.num_pages, 1, 128, n + width), "latent_pages"),
                                    self._cache_needs[0], (torch.int32, (self.total_q,), "positions")))
        _check(_lib.msa_latent_append(self._h, rope and rope._h, _ptr(positions), latent.data_ptr(), strides[0],
                                      key.data_ptr(), strides[1], kv_indices.data_ptr(), n, width,
                                      latent_pages.data_ptr(), _stream(stream)), "msa_latent_append")
        if known is None:
            self._passes("latent_append", tensors, strides)

    def latent_expand(self, latent_pages, w_k, w_v, kv_indices, k_pages, v_pages, stream=None):
        """K and V pages [P, Hkv, 128, d] out of a latent cache's (msa_latent_expand):
        w_k [Hkv, d - rope_dim, latent_dim] and w_v [Hkv, d, latent_dim] bf16."""
        n = w_v.shape[-1]
        width = latent_pages.shape[-1] - n
        tensors = (kv_indices, k_pages, v_pages, latent_pages, w_k, w_v)
        known = self._passed("latent_expand", tensors)
        if not known:
            _need_all(tensors, self._cache_needs[:3] + (
                (torch.bfloat16, (self.num_pages, 1, 128, n + width), "latent_pages"),
                (torch.bfloat16, (self.hkv, self.d - width, n), "w_k"), (torch.bfloat16, (self.hkv, self.d, n), "w_v")))
        _check(_lib.msa_latent_expand(self._h, latent_pages.data_ptr(), w_k.data_ptr(), w_v.data_ptr(),
                                      kv_indices.data_ptr(), n, width, k_pages.data_ptr(), v_pages.data_ptr(),
                                      _stream(stream)), "msa_latent_expand")
        if not known:
            self._passes("latent_expand", tensors)

    # -- stage 1
    def proxy_maxscore(self, pq, pk_pages, kv_indices, out=None, stream=None):
        _need(pq, torch.bfloat16, (self.total_q, self.hp, self.dp), "pq")
        _need(pk_pages, torch.bfloat16, (self.num_pages, 1, 128, self.dp), "pk_pages")
        _need(kv_indices, torch.int32, (self.n_page_entries,), "kv_indices")
        if out is None:
            out = torch.empty((self.n_tiles, self.hp, self.max_blocks), dtype=torch.float32, device=pq.device)
        _need(out, torch.float32, (self.n_tiles, self.hp, self.max_blocks), "max_score")
        _check(_lib.msa_proxy_maxscore(self._h, _ptr(pq), _ptr(pk_pages), _ptr(kv_indices), _ptr(out),
                                       _stream(stream)), "msa_proxy_maxscore")
        return out

    def proxy_maxscore_fp8(self, pq, pk_pages, pk_scale, kv_indices, out=None, stream=None):
        """Decode proxy pass over e4m3 proxy K pages with one fp32 scale
        (msa_proxy_maxscore_fp8)."""
        _need(pq, torch.bfloat16, (self.total_q, self.hp, self.dp), "pq")
        _need(pk_pages, torch.float8_e4m3fn, (self.num_pages, 1, 128, self.dp), "pk_pages")
        _need(pk_scale, torch.float32, (1,), "pk_scale")
        _need(kv_indices, torch.int32, (self.n_page_entries,), "kv_indices")
        if out is None:
            out = torch.empty((self.n_tiles, self.hp, self.max_blocks), dtype=torch.float32, device=pq.device)
        _need(out, torch.float32, (self.n_tiles, self.hp, self.max_blocks), "max_score")
        _check(_lib.msa_proxy_maxscore_fp8(self._h, _ptr(pq), _ptr(pk_pages), _ptr(pk_scale), _ptr(kv_indices),
                                           _ptr(out), _stream(stream)), "msa_proxy_maxscore_fp8")
        return out

    def proxy_maxscore_nvfp4(self, pq, pk_codes, pk_block_scales, pk_global_scale, kv_indices, out=None,
                             stream=None):
        """Decode proxy pass over an NVFP4 proxy K (msa_proxy_maxscore_nvfp4):
        uint8 e2m1 code pairs [P, 1, 128, dp/2], e4m3 block scales [P, 1, 128,
        dp/16] and one fp32 global scale."""
        _need(pq, torch.bfloat16, (self.total_q, self.hp, self.dp), "pq")
        _need(pk_codes, torch.uint8, (self.num_pages, 1, 128, self.dp // 2), "pk_codes")
        _need(pk_block_scales, torch.float8_e4m3fn, (self.num_pages, 1, 128, self.dp // 16), "pk_block_scales")
        _need(pk_global_scale, torch.float32, (1,), "pk_global_scale")
        _need(kv_indices, torch.int32, (self.n_page_entries,), "kv_indices")
        if out is None:
            out = torch.empty((self.n_tiles, self.hp, self.max_blocks), dtype=torch.float32, device=pq.device)
        _need(out, torch.float32, (self.n_tiles, self.hp, self.max_blocks), "max_score")
        _check(_lib.msa_proxy_maxscore_nvfp4(self._h, _ptr(pq), _ptr(pk_codes), _ptr(pk_block_scales),
                                             _ptr(pk_global_scale), _ptr(kv_indices), _ptr(out), _stream(stream)),
               "msa_proxy_maxscore_nvfp4")
        return out

    def proxy_topk(self, pq, pk_pages, kv_indices, out=None, max_score=None, stream=None):
        """Stages 1 and 2 in one launch (msa_proxy_topk): the kv_block_indexes
        msa_topk_select would pick from this plan's proxy scores; max_score,
        when given, receives those scores too."""
        _need(pq, torch.bfloat16, (self.total_q, self.hp, self.dp), "pq")
        _need(pk_pages, torch.bfloat16, (self.num_pages, 1, 128, self.dp), "pk_pages")
        _need(kv_indices, torch.int32, (self.n_page_entries,), "kv_indices")
        if out is None:
            out = torch.empty((self.n_tiles, self.hp, self.topk), dtype=torch.int32, device=pq.device)
        _need(out, torch.int32, (self.n_tiles, self.hp, self.topk), "kv_block_indexes")
        if max_score is not None:
            _need(max_score, torch.float32, (self.n_tiles, self.hp, self.max_blocks), "max_score")
        _check(_lib.msa_proxy_topk(self._h, _ptr(pq), _ptr(pk_pages), _ptr(kv_indices), _ptr(max_score), _ptr(out),
                                   _stream(stream)), "msa_proxy_topk")
        return out

    # -- stage 3
    def sparse_attn(self, q, k_pages, v_pages, kv_indices, kv_block_indexes, k_scale=None, v_scale=None,
                    out=None, lse=None, want_lse=True, stream=None):
        _need_all((kv_indices, k_pages, v_pages, q, kv_block_indexes) if self.kv_dtype == "bf16" else
                  (kv_indices, k_pages, v_pages, k_scale, v_scale, q, kv_block_indexes), self._attn_needs)
        if out is None:
            out = torch.empty_like(q)
        else:
            _need(out, torch.bfloat16, self._q_shape, "out")
        if lse is not None:
            _need(lse, torch.float32, self._lse_shape, "lse")
        elif want_lse:
            lse = torch.empty(self._lse_shape, dtype=torch.float32, device=q.device)
        _check(_lib.msa_sparse_attn(self._h, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                    kv_indices.data_ptr(), kv_block_indexes.data_ptr(), _ptr(k_scale), _ptr(v_scale),
                                    out.data_ptr(), _ptr(lse), _stream(stream)), "msa_sparse_attn")
        return out, lse

    # A step's calls come with tensors like the last step's: what the checks found holds for all of one
    # type, dtype, device, sizes and strides, and comparing those takes a quarter of the checks' time
    # (a call of eight tensors 11.1 -> 8.7 us).  Noted once the library has accepted the call: the tensors
    # are then on the plan's device, which it has found to be the current one.
    def _passed(self, call, tensors):
        known = self._alike.get((call, len(tensors)))
        return known[1] if known is not None and known[0].check(*tensors) else None

    def _passes(self, call, tensors, found=True):
        global _Alike
        if _Alike is None or len({*map(id, tensors)}) < len(tensors):  # (one tensor twice: no comparison lets that pass)
            return
        try:
            alike = _Alike(*tensors, dynamic_dims_sizes=None, dynamic_dims_strides=None)
        except TypeError:  # a torch that makes it in another way
            _Alike = None
            return
        self._alike[call, len(tensors)] = alike, found

    def _outputs(self, out, lse, shape, want_lse):
        # (what _new makes is on the current device, which the library then compares with the plan's)
        if out is None:
            out = _new(shape, (shape[1] * shape[2], shape[2], 1), torch.bfloat16)
        else:
            _need(out, torch.bfloat16, shape, "out")
        if lse is not None:
            _need(lse, torch.float32, self._lse_shape, "lse")
        elif want_lse:
            lse = _new(self._lse_shape, (self.hq, 1), torch.float32)
        return out, lse

    def tree_attn(self, q, k_pages, v_pages, kv_indices, kv_block_indexes, tree_mask, k_scale=None, v_scale=None,
                  out=None, lse=None, want_lse=True, stream=None):
        """Attention of drafted tokens over the cache (msa_tree_attn): row i sees
        the keys before the drafts, and draft b of its sequence iff bit b % 32 of
        tree_mask[i, b // 32] is set (int32 [total_q, 4]), of the selected blocks.
        Drafts that cross a page's edge lie in two blocks, of which topk_select
        takes the first by its score: set max_score[t, :, (kv_len - qo_len) // 128]
        to inf before it, so that no draft loses its ancestors."""
        tensors = ((kv_indices, k_pages, v_pages, q, kv_block_indexes, tree_mask) if self.kv_dtype == "bf16" else
                   (kv_indices, k_pages, v_pages, k_scale, v_scale, q, kv_block_indexes, tree_mask))
        known = self._passed("tree_attn", tensors)
        if not known:
            _need_all(tensors, self._tree_needs)
        out, lse = self._outputs(out, lse, self._q_shape, want_lse)
        _check(_lib.msa_tree_attn(self._h, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), kv_indices.data_ptr(),
                                  kv_block_indexes.data_ptr(), tree_mask.data_ptr(), _ptr(k_scale), _ptr(v_scale),
                                  out.data_ptr(), _ptr(lse), _stream(stream)), "msa_tree_attn")
        if not known:
            self._passes("tree_attn", tensors)
        return out, lse

    def latent_attn(self, q, latent_pages, kv_indices, kv_block_indexes, rope_dim, scale, tree_mask=None, out=None,
                    lse=None, want_lse=True, stream=None):
        """Absorbed attention over a latent cache (msa_latent_attn): q [total_q, Hq,
        latent_dim + rope_dim] bf16, out [total_q, Hq, latent_dim]; causal, or by
        tree_mask as tree_attn has it (with the same word on page edges)."""
        width = q.shape[-1]
        if not 0 <= rope_dim < width:
            raise ValueError("rope_dim: %s, rows have %s" % (rope_dim, width))
        tensors = (q, latent_pages, kv_indices, kv_block_indexes)
        if tree_mask is not None:
            tensors += (tree_mask,)
        known = self._passed("latent_attn", tensors)
        if not known:
            _need_all(tensors, ((torch.bfloat16, (self.total_q, self.hq, width), "q"),
                                (torch.bfloat16, (self.num_pages, 1, 128, width), "latent_pages")) + self._table_needs)
        out, lse = self._outputs(out, lse, (self.total_q, self.hq, width - rope_dim), want_lse)
        _check(_lib.msa_latent_attn(self._h, q.data_ptr(), latent_pages.data_ptr(), kv_indices.data_ptr(),
                                    kv_block_indexes.data_ptr(), _ptr(tree_mask), width - rope_dim, rope_dim,
                                    float(scale), out.data_ptr(), _ptr(lse), _stream(stream)), "msa_latent_attn")
        if not known:
            self._passes("latent_attn", tensors)
        return out, lse

    # -- training extension
    def sparse_attn_bwd(self, q, k_pages, v_pages, kv_indices, kv_block_indexes, out, lse, dout, pq, pk_pages,
                        kl_weight=1.0, grads=None, stream=None):
        _need(dout, torch.bfloat16, tuple(q.shape), "dout")
        _need(out, torch.bfloat16, tuple(q.shape), "out")
        _need(lse, torch.float32, (self.total_q, self.hq), "lse")
        _need(pq, torch.bfloat16, (self.total_q, self.hp, self.dp), "pq")
        _need(pk_pages, torch.bfloat16, (self.num_pages, 1, 128, self.dp), "pk_pages")
        _need(kv_block_indexes, torch.int32, (self.n_tiles, self.hp, self.topk), "kv_block_indexes")
        dev = q.device
        if grads is None:
            grads = dict(dq=torch.empty(q.shape, dtype=torch.float32, device=dev),
                         dk=torch.zeros(k_pages.shape, dtype=torch.float32, device=dev),
                         dv=torch.zeros(v_pages.shape, dtype=torch.float32, device=dev),
                         dpq=torch.empty(pq.shape, dtype=torch.float32, device=dev),
                         dpk=torch.zeros(pk_pages.shape, dtype=torch.float32, device=dev))
        _check(_lib.msa_sparse_attn_bwd(self._h, _ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(kv_indices),
                                        _ptr(kv_block_indexes), _ptr(out), _ptr(lse), _ptr(dout), _ptr(pq),
                                        _ptr(pk_pages), float(kl_weight), _ptr(grads["dq"]), _ptr(grads["dk"]),
                                        _ptr(grads["dv"]), _ptr(grads["dpq"]), _ptr(grads["dpk"]),
                                        _stream(stream)), "msa_sparse_attn_bwd")
        return grads

    def check_errors(self, stream=None):
        _check(_lib.msa_check_errors(self._h, _stream(stream)), "msa_check_errors")


def _device_view_int32(ptr, n, device_index, owner):
    """Wrap a device int32 array owned by libmsa as a torch tensor without
    copying; the tensor and its views keep `owner`, whose memory it is."""
    class _Holder:
        pass
    h = _Holder()
    h.owner = owner
    h.__cuda_array_interface__ = {"shape": (n,), "typestr": "<i4", "data": (ptr, False), "version": 3,
                                  "strides": None}
    with torch.cuda.device(device_index):
        return torch.as_tensor(h, device="cuda:%d" % device_index)
