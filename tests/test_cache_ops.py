"""Rotary positions and the cache appends without a GPU: the oracle's own
definitions against other routes, and the calls' refusals."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import msa_oracle as O

UNSUPPORTED, INVALID = 2, 1


# ------------------------------------------------------------------ oracle --

@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_as_complex_rotation(layout):
    """Pairs as complex numbers times exp(i f pos), dims behind them untouched,
    scores of two rotated heads a function of the positions' difference."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64))
    pos = np.array([0, 1, 7, 1000, 131071])
    f, m = O.rope_freqs(48)
    got = O.rope(x, pos, 48, layout)
    a, b = (x[..., :24], x[..., 24:48]) if layout == "half" else (x[..., 0:48:2], x[..., 1:48:2])
    z = (a + 1j * b) * np.exp(1j * pos[:, None] * f)[:, None]
    ga, gb = (got[..., :24], got[..., 24:48]) if layout == "half" else (got[..., 0:48:2], got[..., 1:48:2])
    assert np.abs(ga - z.real).max() < 1e-9 and np.abs(gb - z.imag).max() < 1e-9 and m == 1.0
    assert np.array_equal(got[..., 48:], x[..., 48:])
    q, k = x[:1], x[1:2]
    one = [float((O.rope(q, [i + 9], 64, layout) * O.rope(k, [i], 64, layout)).sum()) for i in (0, 5, 4000)]
    assert max(one) - min(one) < 1e-9


def test_rope_inverse_is_the_transpose():
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((2, 4, 2, 32))
    kw = dict(scaling="yarn", factor=4.0, original_len=4096)
    pos = [3, 77, 5000, 12]
    lhs = (O.rope(x, pos, 32, **kw) * y).sum()
    assert abs(lhs - (x * O.rope(y, pos, 32, inverse=True, **kw)).sum()) < 1e-9
    m = 0.1 * math.log(4.0) + 1.0
    back = O.rope(O.rope(x, pos, 32, **kw), pos, 32, inverse=True, **kw)
    assert np.abs(back - m * m * x).max() < 1e-9


def test_rope_scalings_closed_form():
    f, _ = O.rope_freqs(64)
    assert np.allclose(O.rope_freqs(64, scaling="linear", factor=8.0)[0], f / 8)
    ntk = O.rope_freqs(64, scaling="ntk", factor=8.0)[0]
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], f[-1] / 8)      # the slowest pair is interpolated, the fastest kept
    yarn, m = O.rope_freqs(64, scaling="yarn", factor=8.0, original_len=4096)
    turns = 4096 * f / (2 * math.pi)
    assert np.allclose(yarn[turns > 64], f[turns > 64]) and np.allclose(yarn[turns < 0.5], f[turns < 0.5] / 8)
    assert (yarn <= f).all() and (yarn >= f / 8).all() and np.isclose(m, 0.1 * math.log(8) + 1)


def test_e4m3_encode_against_torch():
    rng = np.random.default_rng(2)
    x = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.integers(-4, 3, 4000), O.e4m3_to_f64(np.arange(127))])
    x = np.concatenate([x, -x, [0.0, 464.0, 1e30, 2.0 ** -10, 3 * 2.0 ** -10]]).astype(np.float32)
    ref = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.to_e4m3(x), ref)
    assert O.to_e4m3(np.array([np.nan]))[0] & 0x7F == 0x7F


def test_nvfp4_encode_nearest():
    """Decoded values are nowhere further from x than any other code's."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((20, 64)) * 3
    x[0] = 0.0
    x[1, :16] = 1e-9
    g = 8.0 / (448 * 6)
    codes, sc = O.to_nvfp4(x, g)
    got = O.nvfp4_to_f64(codes, sc, g)
    by = np.repeat(O.e4m3_to_f64(sc), 16, axis=-1) * g
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    best = np.abs(np.abs(x)[..., None] - grid * by[..., None]).min(-1)
    assert np.allclose(np.abs(got - x), best, atol=1e-15)
    assert (got[0] == 0).all() and (got[1, :16] == 0).all()


def test_block_scale_borders():
    for e in (-40, -7, 0, 13):
        s = 2.0 ** e
        assert O.block_scale(448 * s) == s
        assert O.block_scale(np.nextafter(448 * s, np.inf)) == 2 * s
    assert O.block_scale(0.0) == 2.0 ** -40 and O.block_scale(1e30) == 2.0 ** 40


def test_append_in_pieces_or_at_once():
    """A page filled row by row holds the codes of the page filled at once, as
    long as no value falls below the smallest step of the last scale."""
    rng = np.random.default_rng(4)
    x = rng.standard_normal((100, 1, 64)) * np.linspace(0.1, 40, 100)[:, None, None]
    x[np.abs(x) < 2.0 ** -4] = 1.0
    empty, sc = np.zeros((1, 1, 128, 64), np.uint8), np.zeros((1, 1))
    whole, s1 = O.kv_append(x, empty, [0], [100], [100], "e4m3_block", sc)
    pages, s2 = empty, sc
    for i in range(100):
        pages, s2 = O.kv_append(x[i:i + 1], pages, [0], [1], [i + 1], "e4m3_block", s2)
    assert s1 == s2
    err = np.abs(O.e4m3_to_f64(pages) - O.e4m3_to_f64(whole))
    assert (err <= 2.0 ** -4 * np.abs(O.e4m3_to_f64(whole))).all()


# ---------------------------------------------------------------- refusals --

@pytest.fixture(scope="module")
def msa():
    try:
        from block_sparse_long_proxy_gb300 import msa
    except ImportError:
        import __graft_entry__
        __graft_entry__.build()
        from block_sparse_long_proxy_gb300 import msa
    return msa


@pytest.mark.parametrize("kw, status", [
    (dict(rotary_dim=8), UNSUPPORTED), (dict(rotary_dim=24), UNSUPPORTED), (dict(rotary_dim=272), UNSUPPORTED),
    (dict(rotary_dim=0), UNSUPPORTED), (dict(rotary_dim=64, base=1.0), INVALID),
    (dict(rotary_dim=64, base=float("nan")), INVALID), (dict(rotary_dim=64, base=float("inf")), INVALID),
    (dict(rotary_dim=64, scaling="linear", factor=0.5), INVALID),
    (dict(rotary_dim=64, scaling="ntk", factor=float("nan")), INVALID),
    (dict(rotary_dim=64, scaling="yarn", factor=4.0), INVALID),               # original_len
    (dict(rotary_dim=64, scaling="yarn", factor=4.0, original_len=4096, beta_fast=1.0, beta_slow=2.0), INVALID),
    (dict(rotary_dim=64, scaling="yarn", factor=4.0, original_len=4096, beta_slow=0.0), INVALID)])
def test_rope_create_refusals(msa, kw, status):
    with pytest.raises(msa.MsaError) as e:
        msa.Rope(**kw)
    assert e.value.status == status


def test_rope_apply_refusals(msa):
    """Every check answers before any device work (no GPU here): the pointers
    are numbers."""
    f, rope = msa._lib, msa.Rope(64)
    base = 1 << 20

    def call(x=base, xs=256, pos=base, n=4, heads=2, d=128, dtype=0, out=2 * base, os=256, h=rope._h):
        return f.msa_rope_apply(h, ctypes.c_void_p(x), xs, ctypes.c_void_p(pos), n, heads, d, dtype, 0,
                                ctypes.c_void_p(out), os, None)
    assert call(n=0) == 0
    assert call(h=None) == INVALID
    for kw in (dict(x=None), dict(pos=None), dict(out=None), dict(n=-1), dict(heads=0), dict(d=0), dict(dtype=2),
               dict(xs=255), dict(xs=248), dict(os=128), dict(x=base + 8), dict(out=2 * base + 2), dict(xs=260),
               dict(d=32, heads=8), dict(out=base + 16), dict(out=base + 512), dict(out=base, os=512),
               dict(x=base, out=base + 256, xs=512, os=512)):
        assert call(**kw) == INVALID, kw
    assert call(d=136, heads=1) == UNSUPPORTED and call(d=272, heads=1, xs=272, os=272) == UNSUPPORTED


def test_append_null_refusals(msa):
    f = msa._lib
    assert f.msa_kv_append(None, None, None, None, 0, None, 0, None, None, None, None, None, None) == INVALID
    assert f.msa_pk_append(None, None, None, None, 0, None, None, None, None, None, None, None, None) == INVALID
    assert f.msa_append_bwd(None, None, None, None, None, None, None, None, None, None, None, None) == INVALID
    f.msa_rope_destroy(None)


@pytest.mark.parametrize("pages, hkv", [(2 ** 21 + 1, 8), (2 ** 24, 2), (2 ** 24 // 3 + 1, 3)])
def test_block_plan_pool_within_32_bit_rows(msa, pages, hkv):
    """K/V rows are addressed in 32 bits: a pool of more is refused (before any
    device work)."""
    with pytest.raises(msa.MsaError) as e:
        one = (ctypes.c_int32 * 1)(1)
        h = ctypes.c_void_p()
        msa._check(msa._lib.msa_plan(one, one, 1, hkv, hkv, hkv, 64, 64, 128, 1, pages, msa.KV_FP8_E4M3_BLOCK, 0, None,
                                     ctypes.byref(h)), "msa_plan")
    assert e.value.status == INVALID
