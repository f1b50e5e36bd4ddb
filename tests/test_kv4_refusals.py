"""The 4-bit paged cache's refusals and sizes, on their arguments alone (no GPU)."""
import ctypes

import numpy as np
import pytest

from oracle import kv4 as ref


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
    return nm.lib().nm_kv4_append(ctypes.byref(c), layer, None, starts, n, T, k, ks, v, vs, q, qs, H, o, os_, rope, rows, None)


def attend(nm, c, layer=0, starts=None, n=1, T=1, most=1, q=P, qs=512, H=4, o=P, os_=512, lse=None):
    return nm.lib().nm_kv4_attention(ctypes.byref(c), layer, None, starts, n, T, most, q, qs, H, 0.1, o, os_, lse, None)


def test_sizes(nm):
    L = nm.lib()
    assert L.nm_kv4_page_bytes(64, 32, 8, 128) == 32 * 8 * 64 * 144
    assert L.nm_kv4_page_bytes(16, 1, 1, 64) == 16 * 72
    for bad in ((8, 1, 1, 128), (48, 1, 1, 128), (64, 0, 1, 128), (64, 1, 0, 128), (64, 1, 1, 96), (256, 1, 1, 128)):
        assert L.nm_kv4_page_bytes(*bad) == 0
    assert L.nm_kv4_workspace_bytes(10, 128) > 0 and L.nm_kv4_workspace_bytes(-1, 128) == 0
    assert L.nm_kv4_workspace_bytes(1, 100) == 0
    # the struct mirrors the header: a pointer, an int64, six int32, five pointers, an int64
    assert ctypes.sizeof(nm.NmKv4Cache) == 8 + 8 + 6 * 4 + 5 * 8 + 8


@pytest.mark.parametrize("field,value,status", [
    ("page_tokens", 24, "UNSUPPORTED"), ("head_dim", 80, "UNSUPPORTED"), ("n_layers", 0, "UNSUPPORTED"),
    ("n_kv_heads", -1, "UNSUPPORTED"), ("n_pages", -1, "SHAPE"), ("max_pages", 1 << 30, "SHAPE"), ("max_seqs", -1, "SHAPE"),
    ("info", None, "INVALID_ARG"), ("lens", None, "INVALID_ARG"), ("refs", None, "INVALID_ARG"), ("tables", None, "INVALID_ARG"),
    ("workspace", None, "INVALID_ARG"), ("pool", None, "INVALID_ARG"), ("pool", P + 64, "ALIGN"), ("refs", P + 4, "ALIGN"),
    ("workspace", P + 128, "ALIGN"), ("workspace_bytes", 100, "SHAPE")])
def test_cache_refusals(nm, field, value, status):
    c = cache(nm, **{field: value})
    want = getattr(nm, "NM_ERR_" + status)
    assert append(nm, c) == want and attend(nm, c) == want
    assert nm.lib().nm_kv4_compact(ctypes.byref(c), None) == want
    if field != "pool" or value is not None:
        assert nm.lib().nm_kv4_reserve(ctypes.byref(c), None, None, 1, None) == want


def test_call_refusals(nm):
    L, c = nm.lib(), cache(nm)
    r = ctypes.byref(c)
    assert append(nm, c, layer=2) == nm.NM_ERR_SHAPE and append(nm, c, layer=-1) == nm.NM_ERR_SHAPE
    assert append(nm, c, T=2) == nm.NM_ERR_SHAPE  # no starts: one token each
    assert append(nm, c, n=-1, T=-1) == nm.NM_ERR_INVALID_ARG
    assert append(nm, c, n=1025, T=1025) == nm.NM_ERR_UNSUPPORTED
    assert append(nm, c, k=None) == nm.NM_ERR_INVALID_ARG and append(nm, c, v=None) == nm.NM_ERR_INVALID_ARG
    assert append(nm, c, k=P + 8) == nm.NM_ERR_ALIGN and append(nm, c, rope=P + 4) == nm.NM_ERR_ALIGN
    assert append(nm, c, ks=248) == nm.NM_ERR_SHAPE and append(nm, c, vs=260) == nm.NM_ERR_SHAPE
    assert append(nm, c, o=None) == nm.NM_ERR_INVALID_ARG and append(nm, c, os_=504) == nm.NM_ERR_SHAPE
    assert append(nm, c, os_=520) == nm.NM_ERR_SHAPE  # q in place with another stride
    assert append(nm, c, rows=-1) == nm.NM_ERR_SHAPE
    assert attend(nm, c, layer=2) == nm.NM_ERR_SHAPE and attend(nm, c, H=3) == nm.NM_ERR_SHAPE
    assert attend(nm, c, H=0) == nm.NM_ERR_SHAPE and attend(nm, c, H=130, qs=1 << 20, os_=1 << 20) == nm.NM_ERR_UNSUPPORTED
    assert attend(nm, c, most=0) == nm.NM_ERR_INVALID_ARG and attend(nm, c, q=None) == nm.NM_ERR_INVALID_ARG
    assert attend(nm, c, o=P + 2) == nm.NM_ERR_ALIGN and attend(nm, c, lse=P + 4) == nm.NM_ERR_ALIGN
    assert attend(nm, c, qs=508) == nm.NM_ERR_SHAPE
    assert L.nm_kv4_fork(r, None, P, 1, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_kv4_fork(r, P, P, -1, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_kv4_free(r, P, 1025, None) == nm.NM_ERR_UNSUPPORTED
    assert L.nm_kv4_read(r, 5, None, None, 1, 1, P, P, 0, None) == nm.NM_ERR_SHAPE
    assert L.nm_kv4_read(r, 0, None, None, 1, 1, P + 2, P, 0, None) == nm.NM_ERR_ALIGN
    other = cache(nm, n_layers=3)
    assert L.nm_kv4_copy_pages(r, P, ctypes.byref(other), P, 1, None) == nm.NM_ERR_SHAPE
    assert L.nm_kv4_copy_pages(r, None, r, P, 1, None) == nm.NM_ERR_INVALID_ARG
    assert L.nm_kv4_init(None, None) == nm.NM_ERR_INVALID_ARG
    # nothing to do
    assert append(nm, c, n=0, T=0) == nm.NM_OK and attend(nm, c, n=0, T=0) == nm.NM_OK
    assert L.nm_kv4_free(r, None, 0, None) == nm.NM_OK


# --- the references themselves -----------------------------------------------------------

def test_quantise_is_near_and_exact_where_it_can_be():
    """Every value is within half a step (one, at the ends) plus the parameters' rounding; sixteen evenly
    spaced values come back exactly; equal channels give their fp16 value."""
    r = np.random.RandomState(0)
    x = (r.randn(50, 2, 128) * np.exp(r.randn(50, 2, 1))).astype(np.float32)
    k, v = ref.quantise(x, x)
    g = x.reshape(50, 2, 2, 64)
    step = (g.max(-1) - g.min(-1)) / 15
    # s is rounded to 2^-9, so the ends are off by 15 s 2^-9 / 2 more; mid by 2^-11 of it
    tol = step * (0.5 + 8 * 2.0 ** -8) + np.abs(g).max(-1) * 2.0 ** -10
    assert np.all(np.abs(k.reshape(g.shape) - g) <= tol[..., None])
    np.testing.assert_array_equal(k, v)
    y = np.tile(np.arange(-8, 8, dtype=np.float32) * 0.25, 8).reshape(1, 1, 128)
    np.testing.assert_array_equal(ref.quantise(y, y)[0], y)
    z = np.full((1, 1, 64), 2.75, np.float32)
    np.testing.assert_array_equal(ref.quantise(z, -z)[1], -z)


def test_attention_reference_against_direct_sums():
    r = np.random.RandomState(1)
    q, K, V = r.randn(3, 4, 8), r.randn(7, 2, 8), r.randn(7, 2, 8)
    out, lse, _, _ = ref.attention(q, K, V, 7, 0.3)
    for i in range(3):
        for h in range(4):
            w = np.array([np.exp(0.3 * sum(q[i, h, d] * K[t, h // 2, d] for d in range(8))) for t in range(7 - 3 + i + 1)])
            np.testing.assert_allclose(out[i, h], (w[:, None] * V[:len(w), h // 2]).sum(0) / w.sum(), rtol=1e-12)
            np.testing.assert_allclose(lse[i, h], np.log(w.sum()), rtol=1e-12)


def test_pages_reference_keeps_its_invariants():
    r = np.random.RandomState(2)
    m = ref.Pages(30, 16, 6, 8)
    for _ in range(300):
        ids = r.permutation(6)[:r.randint(1, 4)].tolist()
        if r.rand() < 0.5:
            m.reserve(ids, r.randint(0, 40, len(ids)).tolist())
        elif r.rand() < 0.5:
            m.fork([int(r.randint(6)) for _ in ids], ids)
        elif r.rand() < 0.7:
            m.free(ids)
        else:
            m.compact()
        named = [p for t in m.tables for p in t if p >= 0]
        assert [named.count(p) for p in range(30)] == m.refs
        for t, n in zip(m.tables, m.lens):
            assert sum(p >= 0 for p in t) == -(-n // 16)
            if n % 16:
                assert m.refs[t[n // 16]] == 1, "a partial page has one owner"
