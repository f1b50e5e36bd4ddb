"""The 8-bit paged cache's refusals and sizes, on their arguments alone (no GPU)."""
import ctypes

import numpy as np
import pytest

from oracle import kv8 as ref


@pytest.fixture(scope="module")
def nm():
    from sparse_decoding_gb300 import build
    build.build()
    import sparse_decoding_gb300 as nm
    nm.lib()
    return nm


_buf = (ctypes.c_uint8 * 8192)()
P = (ctypes.addressof(_buf) + 255) & ~255


def cache(nm, **kw):
    f = dict(pool=P, n_pages=4, page_tokens=32, n_layers=2, n_kv_heads=2, head_dim=128, max_seqs=3, max_pages=4, info=P,
             lens=P, refs=P, tables=P, workspace=P, workspace_bytes=1 << 40)
    f.update(kw)
    return nm.NmKv4Cache(*[f[n] for n, _ in nm.NmKv4Cache._fields_])


def append(nm, c, layer=0, starts=None, n=1, T=1, k=P, ks=256, v=P, vs=256, q=P, qs=512, H=4, o=P, os_=512, rope=P, rows=9):
    return nm.lib().nm_kv8_append(ctypes.byref(c), layer, None, starts, n, T, k, ks, v, vs, q, qs, H, o, os_, rope, rows, None)


def attend(nm, c, layer=0, starts=None, n=1, T=1, most=1, q=P, qs=512, H=4, scale=0.1, pages=None, m=0, o=P, os_=512, lse=None):
    return nm.lib().nm_kv8_attention(ctypes.byref(c), layer, None, starts, n, T, most, q, qs, H, scale, pages, m, o, os_, lse, None)


def select(nm, c, layer=0, starts=None, n=1, T=1, q=P, qs=512, H=4, m=4, first=1, last=1, pages=P):
    return nm.lib().nm_kv8_select(ctypes.byref(c), layer, None, starts, n, T, q, qs, H, m, first, last, pages, None)


def test_sizes(nm):
    L = nm.lib()
    assert L.nm_kv8_page_bytes(64, 32, 8, 128) == 32 * 8 * (4 * (32 * 128 + 16) + 2 * 128 + 16)
    assert L.nm_kv8_page_bytes(16, 1, 1, 64) == 32 * 64 + 16 + 2 * 64 + 16
    for bad in ((8, 1, 1, 128), (48, 1, 1, 128), (64, 0, 1, 128), (64, 1, 0, 128), (64, 1, 1, 96), (256, 1, 1, 128)):
        assert L.nm_kv8_page_bytes(*bad) == 0
    assert L.nm_kv8_workspace_bytes(10, 128) > 0 and L.nm_kv8_workspace_bytes(-1, 128) == 0
    assert L.nm_kv8_workspace_bytes(1, 100) == 0


@pytest.mark.parametrize("field,value,status", [
    ("page_tokens", 24, "UNSUPPORTED"), ("head_dim", 80, "UNSUPPORTED"), ("n_layers", 0, "UNSUPPORTED"),
    ("n_pages", -1, "SHAPE"), ("max_pages", 1 << 30, "SHAPE"), ("max_seqs", -1, "SHAPE"),
    ("info", None, "INVALID_ARG"), ("lens", None, "INVALID_ARG"), ("refs", None, "INVALID_ARG"), ("tables", None, "INVALID_ARG"),
    ("workspace", None, "INVALID_ARG"), ("pool", None, "INVALID_ARG"), ("pool", P + 64, "ALIGN"), ("refs", P + 4, "ALIGN"),
    ("workspace", P + 128, "ALIGN"), ("workspace_bytes", 100, "SHAPE")])
def test_cache_refusals(nm, field, value, status):
    c = cache(nm, **{field: value})
    want = getattr(nm, "NM_ERR_" + status)
    assert append(nm, c) == want and attend(nm, c) == want and select(nm, c) == want
    assert nm.lib().nm_kv8_compact(ctypes.byref(c), None) == want
    if field != "pool" or value is not None:
        assert nm.lib().nm_kv8_reserve(ctypes.byref(c), None, None, 1, None) == want
        assert nm.lib().nm_kv8_init(ctypes.byref(c), None) == want


def test_call_refusals(nm):
    L, c = nm.lib(), cache(nm)
    r = ctypes.byref(c)
    assert append(nm, c, layer=2) == nm.NM_ERR_SHAPE and append(nm, c, T=2) == nm.NM_ERR_SHAPE
    assert append(nm, c, n=-1, T=-1) == nm.NM_ERR_INVALID_ARG and append(nm, c, n=1025, T=1025) == nm.NM_ERR_UNSUPPORTED
    assert append(nm, c, k=None) == nm.NM_ERR_INVALID_ARG and append(nm, c, k=P + 8) == nm.NM_ERR_ALIGN
    assert append(nm, c, ks=248) == nm.NM_ERR_SHAPE and append(nm, c, os_=520) == nm.NM_ERR_SHAPE
    assert append(nm, c, rope=P + 4) == nm.NM_ERR_ALIGN and append(nm, c, rows=-1) == nm.NM_ERR_SHAPE
    assert attend(nm, c, layer=2) == nm.NM_ERR_SHAPE and attend(nm, c, H=3) == nm.NM_ERR_SHAPE
    assert attend(nm, c, H=130, qs=1 << 20, os_=1 << 20) == nm.NM_ERR_UNSUPPORTED
    assert attend(nm, c, most=0) == nm.NM_ERR_INVALID_ARG and attend(nm, c, scale=float("nan")) == nm.NM_ERR_INVALID_ARG
    assert attend(nm, c, scale=float("inf")) == nm.NM_ERR_INVALID_ARG and attend(nm, c, lse=P + 4) == nm.NM_ERR_ALIGN
    assert attend(nm, c, pages=P, m=0) == nm.NM_ERR_INVALID_ARG and attend(nm, c, pages=P + 2, m=1) == nm.NM_ERR_ALIGN
    assert attend(nm, c, pages=P, m=49153) == nm.NM_ERR_UNSUPPORTED
    assert select(nm, c, layer=-1) == nm.NM_ERR_SHAPE and select(nm, c, H=3) == nm.NM_ERR_SHAPE
    assert select(nm, c, q=None) == nm.NM_ERR_INVALID_ARG and select(nm, c, q=P + 8) == nm.NM_ERR_ALIGN
    assert select(nm, c, pages=None) == nm.NM_ERR_INVALID_ARG and select(nm, c, pages=P + 1) == nm.NM_ERR_ALIGN
    assert select(nm, c, m=0) == nm.NM_ERR_INVALID_ARG and select(nm, c, m=49153) == nm.NM_ERR_UNSUPPORTED
    assert select(nm, c, first=-1) == nm.NM_ERR_INVALID_ARG and select(nm, c, last=0) == nm.NM_ERR_INVALID_ARG
    assert select(nm, c, first=3, last=2) == nm.NM_ERR_INVALID_ARG
    assert select(nm, c, first=(1 << 31) - 1, last=1) == nm.NM_ERR_INVALID_ARG
    assert select(nm, cache(nm, max_pages=49153)) == nm.NM_ERR_UNSUPPORTED
    assert L.nm_kv8_fork(r, None, P, 1, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_kv8_free(r, P, 1025, None) == nm.NM_ERR_UNSUPPORTED
    assert L.nm_kv8_read(r, 5, None, None, 1, 1, P, P, 0, None) == nm.NM_ERR_SHAPE
    assert L.nm_kv8_read(r, 0, None, None, 1, 1, P + 2, P, 0, None) == nm.NM_ERR_ALIGN
    other = cache(nm, n_layers=3)
    assert L.nm_kv8_copy_pages(r, P, ctypes.byref(other), P, 1, None) == nm.NM_ERR_SHAPE
    assert L.nm_kv8_copy_pages(r, None, r, P, 1, None) == nm.NM_ERR_INVALID_ARG


# --- the references themselves ----------------------------------------------------------

def test_reference_codes():
    """Every 8-bit float is its own nearest; the middles go to the even one."""
    codes = sorted({m * 2.0 ** -9 for m in range(8)} | {(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)})
    assert codes[-1] == 448 and len(codes) == 127
    x = np.array(codes)
    np.testing.assert_array_equal(ref.e4m3(x), x)
    np.testing.assert_array_equal(ref.e4m3(-x), -x)
    mid = (x[1:] + x[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, x[:-1], x[1:])
    np.testing.assert_array_equal(ref.e4m3(mid), even)
    for nudge, want in ((1 - 1e-9, x[:-1]), (1 + 1e-9, x[1:])):
        np.testing.assert_array_equal(ref.e4m3(mid * nudge), want)


def test_reference_exponents():
    for most, want in ((448.0, 0), (448.1, 1), (224.0, -1), (0.0, -24), (1e-9, -24), (32768.0, 7), (1e9, 7)):
        assert ref.exponent(most, 448.0, -24, 7) == want
    assert ref.exponent(127.0, 127.0, -30, 100) == 0 and ref.exponent(127.5, 127.0, -30, 100) == 1


def test_reference_held_values():
    """The error of a value is half a step of its code; a second rounding changes only what is small."""
    r = np.random.RandomState(0)
    s = ref.Sequence(2, 64)
    k, v = (r.randn(40, 2, 64).astype(np.float32) for _ in range(2))
    s.append(k, v)
    scale = np.exp2(s.e[np.arange(40) // 16, :, 0].astype(float))[..., None]
    assert np.all(np.abs(s.k - k) <= np.maximum(np.abs(k) * 2.0 ** -4, scale * 2.0 ** -10))
    before = s.k.copy()
    s.append(np.full((1, 2, 64), 300.0, np.float32), v[:1])
    grown = np.exp2(s.e[2, :, 0].astype(float))[None, :, None]
    small = np.abs(before[32:]) < 2.0 ** -6 * grown
    assert np.array_equal(s.k[32:40][~small], before[32:][~small]) and np.array_equal(s.k[:32], before[:32])


def test_reference_selection_bounds_the_scores():
    """What select ranks by is above the largest sum of scores of each page, but for q's rounding."""
    r = np.random.RandomState(1)
    K = ref.Sequence(1, 64)
    K.append(r.randn(320, 1, 64).astype(np.float32) * 2, np.zeros((320, 1, 64), np.float32))
    q = r.randn(4, 64)
    p, m = np.maximum(q, 0).sum(0), np.minimum(q, 0).sum(0)
    for z in range(20):
        up, low, step = ref.bounds(K.k[16 * z:16 * z + 16])
        bound = ((p * up[0] + m * low[0]) * step[0]).sum()
        assert bound >= (K.k[16 * z:16 * z + 16, 0] @ q.T).max(0).sum()
    got = ref.select(q.astype(np.float32), K.k, 16, 6, 1, 2)
    assert got.shape == (1, 6) and got[0, 0] == 0 and list(got[0, -2:]) == [18, 19] and np.all(np.diff(got[0]) > 0)


def test_max_new_is_not_looked_at_with_pages(nm):
    """What such a call is refused for is something else of it."""
    c = cache(nm)
    for most in (0, -1, 1):
        assert attend(nm, c, most=most, pages=P + 2, m=1) == nm.NM_ERR_ALIGN
        assert attend(nm, c, most=most, pages=P, m=0) == nm.NM_ERR_INVALID_ARG
        assert attend(nm, c, most=most, pages=P, m=49153) == nm.NM_ERR_UNSUPPORTED
    assert attend(nm, c, most=0, m=1) == nm.NM_ERR_INVALID_ARG


def test_example_refuses_pages_that_it_cannot_select():
    """Before anything is put on a device."""
    from examples import paged_decode as ex
    for kw in (dict(bits=4, pages=2), dict(bits=8, pages=-1)):
        with pytest.raises(ValueError):
            ex.Decoder(**kw)
