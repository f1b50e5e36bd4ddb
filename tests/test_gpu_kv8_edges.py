"""Calls of the 8-bit paged cache at the edges of what its header allows, on a GPU: lists of pages that are not in order,
selection over many pages, values far below their neighbours' and queries far above. Tolerances as in test_gpu_kv8.py."""
import numpy as np
import pytest
import torch

from oracle import kv8 as ref
from tests.test_gpu_kv4 import f32, f64, ints, starts_of, values
from tests.test_gpu_kv8 import make, nm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def right(got, lse, q, K, V, scale, listed=None, P=0, more=0.0):
    """One token's out [H][D] and lse [H] over positions 0 .. len(K) - 1 (those in the listed pages alone): within
    the tolerances; more: what else a channel of out may be off by."""
    K, V = K.astype(np.float64), V.astype(np.float64)
    lists = None if listed is None else np.array(listed, dtype=int).reshape(1, K.shape[1], -1)
    o, l, A, B = ref.attention(f64(q[None]), K, V, len(K), scale, lists, P)
    e = 2.0 ** -16 * B + 2.0 ** -15
    # weights below fp16's normal range: 2^-25 of codes up to 448 under a weight of at least 2^6, with the scale of the heaviest block
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + len(K) * (2.0 ** -30 * np.abs(V).max() + 2.0 ** -46) + more
    seen = np.isfinite(l)
    gl, go = f64(lse[None]), f64(got[None])
    return np.array_equal(np.isneginf(gl), np.isneginf(l)) and np.all(go[~seen] == 0) and \
        np.all(np.abs(gl[seen] - l[seen]) <= e[seen]) and np.all(np.abs(go - o)[seen] <= tol[seen])


def many(Hk):
    """So many tokens that a warp takes each list by itself (kv8_launch_attention: from five lists an SM on)."""
    return -(-5 * torch.cuda.get_device_properties(0).multi_processor_count // Hk) + 3


LISTS = [[0, 3, 9], [1, 4, 2, 4], [1, 1 << 20, 5], [1, -2, 5], [0, -1, 7, 9], [9, 3, 5, 9, 10], [2, 2, 2, 3], [7, "end", 8],
         [-1, 3], [5, 1 << 30, -(1 << 31), 6], [-7, 2, 3], ["last", 3], [0, 1, "last", 2, "last", "end"], [3] + [-1] * 10 + [4]]


@pytest.mark.parametrize("D,P,Hq", [(128, 64, 8), (64, 16, 4), (128, 16, 13)])
@pytest.mark.parametrize("each", [False, True])
def test_entries_that_count(nm, D, P, Hq, each):
    """Lists out of order and range, with good entries behind bad ones and entries behind the end: what counts, and what
    is reported, is the same in the kernel for few lists and in that for many."""
    n, m = 20 * P + 5, 12
    T = many(1) if each else 5
    if n < T + 4 * P:
        n = T + 20 * P
    count = -(-n // P)
    c, held = make(nm, [n], P=P, L=1, Hk=1, D=D, seed=n)
    q = values(T, Hq, D, 7)
    starts = starts_of([T])
    for x in LISTS:
        bad = [{"last": count - 1, "end": count}.get(e, e) for e in x] + [-1] * (m - len(x))
        taken, faults = ref.listed(bad, count)
        pages = torch.full((T, 1, m), -1, dtype=torch.int32, device="cuda")
        pages[:, 0, :3] = ints([0, 1, 2])
        at = [0, T - 1]
        for t in at:
            pages[t, 0] = ints(bad)
        out, lse = c.attention(0, q, starts=starts, pages=pages, lse=True)
        assert nm.device_status() == (nm.NM_ERR_BOUNDS if faults else nm.NM_OK), x
        for t in at:
            k = n - T + t + 1
            assert right(out[t], lse[t], q[t], held[0].k[:k], held[0].v[:k], D ** -0.5, taken or [-1], P), (x, t)
        k = n - T + 2
        assert right(out[1], lse[1], q[1], held[0].k[:k], held[0].v[:k], D ** -0.5, [0, 1, 2], P), x


@pytest.mark.parametrize("D,P,Hk,Hq", [(128, 16, 1, 8), (64, 32, 1, 16)])
@pytest.mark.parametrize("each", [False, True])
def test_long_lists_out_of_order(nm, D, P, Hk, Hq, each):
    """Hundreds of entries, of which an early one decides what counts much later (in another piece of the list)."""
    m = 300
    n = m * P - 3
    T = many(Hk) if each else 3
    c, held = make(nm, [n], P=P, L=1, Hk=Hk, D=D, seed=P)
    q = values(T, Hq, D, 8)
    starts = starts_of([T])
    for at, value in ((40, 250), (0, 299), (299, 298), (170, -5), (100, -1), (250, 3)):
        bad = np.arange(m)
        bad[at] = value
        taken, faults = ref.listed(bad, m)
        pages = torch.zeros(T, Hk, m, dtype=torch.int32, device="cuda")
        pages[:, :, 1:] = -1
        pages[T - 1] = torch.from_numpy(bad.astype(np.int32)).cuda()
        out, lse = c.attention(0, q, starts=starts, pages=pages, lse=True)
        assert nm.device_status() == (nm.NM_ERR_BOUNDS if faults else nm.NM_OK), (at, value)
        assert right(out[T - 1], lse[T - 1], q[T - 1], held[0].k, held[0].v, D ** -0.5, taken, P), (at, value)
        o2, l2 = c.attention(0, q, starts=starts, pages=pages, lse=True)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
        nm.device_status()


def test_lists_of_thousands(nm):
    """A token's list of 3000 pages: in order, and with one entry that decides what counts a thousand later."""
    D, P, m = 64, 16, 3000
    n = m * P
    c, held = make(nm, [n], P=P, L=1, Hk=1, D=D, seed=9)
    q = values(1, 8, D, 10)
    for at, value in ((0, 0), (100, 1500), (1100, 2), (2999, 2998), (2500, -1)):
        bad = np.arange(m)
        bad[at] = value
        taken, faults = ref.listed(bad, m)
        pages = torch.from_numpy(bad.astype(np.int32)).cuda().view(1, 1, m)
        out, lse = c.attention(0, q, pages=pages, lse=True)
        assert nm.device_status() == (nm.NM_ERR_BOUNDS if faults else nm.NM_OK), (at, value)
        assert right(out[0], lse[0], q[0], held[0].k, held[0].v, D ** -0.5, taken, P), (at, value)


def held_cache(nm, k, v, P, extra=1):
    """A cache of one sequence and layer that holds k and v: (cache, ref.Sequence)."""
    n, Hk, D = k.shape
    c = nm.Kv8Cache(-(-n // P) + extra, P, 1, Hk, D, 1, -(-n // P) + extra)
    c.pool.fill_(0xFF)
    c.reserve(starts=ints([0, n]))
    c.append(0, k, v, starts=ints([0, n]))
    h = ref.Sequence(Hk, D)
    h.append(f32(k), f32(v))
    return c, h


@pytest.mark.parametrize("D,small", [(128, 1e-4), (64, 1e-4), (128, 3e-6)])
@pytest.mark.parametrize("max_new", [1, 160])
def test_values_far_below_later_ones(nm, D, small, max_new):
    """The first 64 tokens have small values, the next ones, of the same 128, the largest there are: rows that see the first
    alone are right all the same. Off by at most 2^-32 of the largest scale more in the kernel for prompts."""
    n, H, P = 200, 16, 16
    k, v = values(n, 1, D, 1), values(n, 1, D, 2)
    v[:64] = (v[:64].float() * small).bfloat16()
    v[64:] = (v[64:].float() * 8000).bfloat16()
    c, h = held_cache(nm, k, v, P)
    assert h.e[4, 0, 1] == 7
    q = values(160, H, D, 3)
    out, lse = c.attention(0, q, starts=ints([0, 160]), max_new=max_new, lse=True)
    assert nm.device_status() == nm.NM_OK
    for t in (0, 5, 22, 23, 24, 60, 159):
        m = n - 160 + t + 1
        assert right(out[t], lse[t], q[t], h.k[:m], h.v[:m], D ** -0.5, more=2.0 ** -32 * 128 if max_new > 1 else 0.0), t


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_new", [1, 100, 0])
def test_queries_up_to_the_largest_number(nm, D, max_new):
    """q up to 2^128 with a scale that makes its scores ordinary, in each kernel (0: over lists)."""
    n, H, P = 150, 16, 16
    k, v = values(n, 1, D, 4, 0.01), values(n, 1, D, 5)
    c, h = held_cache(nm, k, v, P)
    g = torch.Generator().manual_seed(6)
    q = (torch.randn(100, H, D, generator=g) * 2.0 ** 126).clamp(-3.3e38, 3.3e38).bfloat16().cuda()
    pages = torch.arange(10, dtype=torch.int32, device="cuda").expand(100, 1, 10).contiguous()
    kw = dict(pages=pages) if max_new == 0 else dict(max_new=max_new)
    out, lse = c.attention(0, q, starts=ints([0, 100]), scale=2.0 ** -126, lse=True, **kw)
    assert nm.device_status() == nm.NM_OK and bool((q.float().abs() > 2.0 ** 127).any())
    for t in (0, 50, 99):
        m = n - 100 + t + 1
        assert right(out[t], lse[t], q[t], h.k[:m], h.v[:m], 2.0 ** -126), t


@pytest.mark.parametrize("max_new", [1, 100, 0])
def test_large_scales_of_scores_that_are_zero(nm, max_new):
    """Keys of zeros: any finite q and scale give even weights."""
    n, H, D, P = 150, 16, 128, 16
    v = values(n, 1, D, 5)
    c, h = held_cache(nm, torch.zeros_like(v), v, P)
    q = (values(100, H, D, 6).float() * 2.0 ** 120).bfloat16()
    q[:, ::2] *= 2.0 ** -130
    pages = torch.arange(10, dtype=torch.int32, device="cuda").expand(100, 1, 10).contiguous()
    kw = dict(pages=pages) if max_new == 0 else dict(max_new=max_new)
    for scale in (2.0 ** 100, -2.0 ** 127, 1.0):
        out, lse = c.attention(0, q, starts=ints([0, 100]), scale=scale, lse=True, **kw)
        for t in (0, 99):
            m = n - 100 + t + 1
            assert right(out[t], lse[t], q[t] * 0, h.k[:m], h.v[:m], 1.0), (scale, t)
    assert nm.device_status() == nm.NM_OK


@pytest.mark.parametrize("pages", [1, 2])
def test_example_with_few_pages(nm, pages):
    """The example's loop with a single page a step, its last one, or the first and the last."""
    from examples import paged_decode as ex
    d = ex.Decoder(layers=1, hidden=256, heads=8, kv_heads=2, dim=64, ffn=512, sequences=2, tokens=80, page=16, seed=5, bits=8, pages=pages)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(8, 256, generator=g, device="cuda").bfloat16()
    trace, one = [], ints([0])
    for _ in range(5):
        trace.append([])
        d.step(x, one, starts=ints([0, 8]), trace=trace[-1])
    rope = d.rope.cpu().numpy()
    h = ref.Sequence(2, 64)
    for step in trace:
        (q, k, v, a), = step
        q, k, v = (f32(t).reshape(8, -1, 64) for t in (q, k, v))
        pos = np.arange(len(h.k), len(h.k) + 8)
        cos, sin = rope[pos, :32], rope[pos, 32:]
        h.append(ref.rotate(k, cos, sin), v)
        q = torch.from_numpy(ref.bf16(ref.rotate(q, cos, sin)))
    for t in range(8):  # of the last step: pages 0 .. 2
        m = len(h.k) - 7 + t
        last = (m - 1) // 16
        K, V = h.k[:m].astype(np.float64), h.v[:m].astype(np.float64)
        lists = np.array([[[last]] * 2 if pages == 1 else [[0, last]] * 2])
        o, _, A, B = ref.attention(f64(q[t:t + 1]), K, V, m, 0.125, lists, 16)
        e = 2.0 ** -16 * B[..., None] + 2.0 ** -15
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e + 2.0 ** -14) * A + 1e-6
        assert np.all(np.abs(f64(a[t]).reshape(o.shape) - o) <= tol), t
    assert nm.device_status() == nm.NM_OK
# --- selection over many pages, whole lists of many query heads, tables ---------------------

@pytest.mark.parametrize("new", [[1], [2], [5]])
def test_select_many_pages_by_a_cluster(nm, new):
    """Head size 128: more pages than the CTAs of a cluster score in one turn of their loop."""
    D, P, n = 128, 16, 40000
    c, held = make(nm, [n], P=P, L=1, Hk=1, D=D, seed=60)
    q = values(new[0], 4, D, 61)
    for m, first, last in ((100, 2, 3), (1999, 0, 1), (2, 1, 1)):
        pages = c.select(0, q, m, starts=starts_of(new), first=first, last=last)
        for t in {0, new[0] - 1}:
            want = ref.select(f32(q[t]), held[0].k[:n - new[0] + t + 1], P, m, first, last)
            np.testing.assert_array_equal(pages[t].cpu().numpy(), want)
    assert nm.device_status() == nm.NM_OK


@pytest.mark.parametrize("D", [64, 128])
def test_select_many_pages_by_a_cta(nm, D):
    """So many tokens and kv heads that each has one CTA, with more pages than it scores in one turn of its loop."""
    P, Hk, n, S = 16, 8, 9000, 40
    c, held = make(nm, [n], P=P, L=1, Hk=Hk, D=D, seed=62)
    q = values(S, 16, D, 63)
    seqs = torch.zeros(S, dtype=torch.int32, device="cuda")  # one sequence, listed often
    for m in (2, 150):
        pages = c.select(0, q, m, seqs=seqs)
        for t in (0, 39):
            np.testing.assert_array_equal(pages[t].cpu().numpy(), ref.select(f32(q[t]), held[0].k, P, m, 1, 1))
    assert nm.device_status() == nm.NM_OK


@pytest.mark.parametrize("new", [[1, 1], [40, 3], [200, 100]])
def test_select_long_sequences(nm, new):
    """Head size 128 and hundreds of pages, by clusters, CTAs and tiles of tokens."""
    D, P, Hk, n = 128, 16, 2, 150
    lens = [9000, 8000]
    c, held = make(nm, lens, P=P, L=1, Hk=Hk, D=D, seed=64)
    q = values(sum(new), 8, D, 65)
    pages = c.select(0, q, n, starts=starts_of(new))
    at = 0
    for s, w in enumerate(new):
        for t in sorted({0, w // 2, w - 1}):
            want = ref.select(f32(q[at + t]), held[s].k[:lens[s] - w + t + 1], P, n, 1, 1)
            np.testing.assert_array_equal(pages[at + t].cpu().numpy(), want)
        at += w
    assert nm.device_status() == nm.NM_OK


@pytest.mark.parametrize("D,tokens,Hq", [(128, 700, 32), (64, 700, 40), (128, 250, 64)])
def test_lists_of_many_query_heads(nm, D, tokens, Hq):
    """More than 16 query heads to a kv head: tiles of a list's rows, more tiles than CTAs, and lists of more than 32
    cells: whole ones, or ones that an even cut goes through."""
    P, n, m = 64, 1500, 9
    c, held = make(nm, [n], P=P, L=1, Hk=1, D=D, seed=66)
    q = values(tokens, Hq, D, 67)
    pages = c.select(0, q, m, starts=starts_of([tokens]))
    pages[3, 0, 1:] = -1
    pages[tokens - 1] = -1
    out, lse = c.attention(0, q, starts=starts_of([tokens]), pages=pages, lse=True)
    for t in (0, 1, 3, tokens // 2, tokens - 2, tokens - 1):
        k = n - tokens + t + 1
        assert right(out[t], lse[t], q[t], held[0].k[:k], held[0].v[:k], D ** -0.5, pages[t].cpu().numpy(), P), t
    o2, l2 = c.attention(0, q, starts=starts_of([tokens]), pages=pages, lse=True)
    assert torch.equal(out, o2) and torch.equal(lse, l2) and nm.device_status() == nm.NM_OK


def test_damaged_tables_are_reported_by_each_kernel(nm):
    """A page that is none of the pool's: each of the attention's kernels reports it and answers another sequence as before."""
    D, P, H = 128, 16, 8
    c, held = make(nm, [1200, 300], P=P, L=1, Hk=1, D=D, seed=68)
    few, some, each = values(2, H, D, 69), values(300, H, D, 70), values(many(1), H, D, 71)
    calls = {"rows": lambda: c.attention(0, few, max_new=1),
             "prompt": lambda: c.attention(0, some, starts=starts_of([200, 100])),
             "lists of few": lambda: c.attention(0, few, pages=lists[:2]),
             "lists of many": lambda: c.attention(0, each, starts=starts_of([each.shape[0] - 100, 100]), pages=lists[2:])}
    lists = torch.cat([c.select(0, few, 5), c.select(0, each, 5, starts=starts_of([each.shape[0] - 100, 100]))])
    good = {x: f() for x, f in calls.items()}
    assert nm.device_status() == nm.NM_OK
    c.tables[1, 18], c.tables[1, 0] = -7, c.n_pages
    for x, f in calls.items():
        bad = f()
        assert nm.device_status() == nm.NM_ERR_BOUNDS, x
        first = 1 if bad.shape[0] == 2 else bad.shape[0] - 100  # rows of sequence 0
        assert torch.equal(bad[:first], good[x][:first]) and bool(torch.isfinite(bad).all()), x
        assert not torch.equal(bad[first:], good[x][first:]), x
    c.select(0, few, 5)
    assert nm.device_status() == nm.NM_ERR_BOUNDS
