"""The 4-bit paged KV cache where rows, pages and parts are not the ordinary ones, on a GPU: joins of many
parts, rows that no sequence covers, pages that are missing. Tolerances as in tests/test_gpu_kv4.py."""
import numpy as np
import pytest
import torch

from oracle import kv4 as ref
from tests.test_gpu_kv4 import f32, f64, ints, make, nm, rope_table, starts_of, values  # noqa: F401

pytestmark = pytest.mark.gpu


def definition(q, K, V, limits, scale):
    """(out, lse, A, B) as oracle.kv4.attention, one matrix product a head: q [n][H][D] (fp64); row i sees the
    tokens of limits[i], a count or a list of truth values."""
    n, H, D = q.shape
    r = H // K.shape[1]
    see = np.zeros((n, len(K)), bool)
    for i, x in enumerate(limits):
        see[i] = x if np.ndim(x) else np.arange(len(K)) < x
    out, A = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, B = np.full((n, H), -np.inf), np.zeros((n, H))
    some = see.any(1)
    for h in range(H):
        k, v = K[:, h // r].astype(np.float64), V[:, h // r].astype(np.float64)
        s = np.where(see, q[:, h] @ k.T * scale, -np.inf)[some]
        if not len(s):
            continue
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        z = p.sum(1, keepdims=True)
        lse[some, h] = (top + np.log(z))[:, 0]
        out[some, h], A[some, h] = p / z @ v, p / z @ np.abs(v)
        B[some, h] = np.where(see, np.abs(q[:, h]) @ np.abs(k).T * abs(scale), 0.0)[some].max(1)
    return out, lse, A, B


def compare(out, lse, want, length, vmax):
    o, l, A, B = want
    e = 2.0 ** -16 * B + 2.0 ** -15
    got, gl = f64(out), lse.cpu().numpy().astype(np.float64)
    seen = np.isfinite(l)
    assert np.array_equal(np.isneginf(gl), ~seen) and np.all(got[~seen] == 0)
    assert np.all(np.abs(gl[seen] - l[seen]) <= e[seen]), np.abs(gl[seen] - l[seen]).max()
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + length * 2.0 ** -30 * vmax + 1e-30
    assert np.all(np.abs(got - o)[seen] <= tol[seen]), (np.abs(got - o)[seen] / tol[seen]).max()


# --- joins of many parts ---------------------------------------------------------------

BLOCK, OVER, MIN_SHARE = 128, 3, 2  # the prompt kernel's: tokens of a block, what a segment adds, blocks of a CTA


def parts_of_first(blocks, others, ctas):
    """CTAs that share the first segment of a line: `blocks` long, others (their blocks) behind it."""
    total = blocks + OVER + sum(n + OVER for n in others)
    share = max(-(-total // ctas), MIN_SHARE + OVER)
    return (OVER + blocks - 1) // share - OVER // share + 1


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("parts", [8, 9, 13, 16, 17, 33, 64, 65, 73, 144, 145])
def test_prompt_attention_joins_many_parts(nm, D, parts):
    """A few new tokens behind a long context beside a short prompt: one segment is cut over 8 CTAs (one
    join) to 145 (groups of parts, then the groups; some with a last group of one part)."""
    H, new = 16, [9, 70]
    others = [1] * 5  # pairs of 16 tokens of the second sequence
    ctas = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    blocks = next((n for n in range(1, 2000) if parts_of_first(n, others, ctas) == parts), None)
    if blocks is None:
        pytest.skip(f"no length gives {parts} parts on {ctas} CTAs")
    lens = [blocks * BLOCK - 5, 70]
    c, K, V = make(nm, lens, P=64, L=1, Hk=1, D=D, seed=parts)
    q = values(sum(new), H, D, 7)
    out, lse = c.attention(0, q, starts=starts_of(new), max_new=70, lse=True)
    assert nm.device_status() == nm.NM_OK
    at = 0
    for s, n in enumerate(new):
        rows = slice(at, at + n)
        want = definition(f64(q[rows]), K[s], V[s], [lens[s] - n + i + 1 for i in range(n)], D ** -0.5)
        compare(out[rows], lse[rows], want, lens[s], np.abs(V[s]).max())
        at += n
    for _ in range(3):  # the counters are as they were, and the order of the sums is fixed
        o2, l2 = c.attention(0, q, starts=starts_of(new), max_new=70, lse=True)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("lens,new,heads", [([30011, 17, 9000], [20, 2, 5], 64), ([30011], [40], 32)])
def test_prompt_attention_long_cut_over_many_ctas(nm, lens, new, heads):
    """Several long segments, each cut over tens of CTAs that end one segment and begin the next."""
    c, K, V = make(nm, lens, P=64, L=1, Hk=1, seed=23)
    q = values(sum(new), heads, 128, 24)
    out, lse = c.attention(0, q, starts=starts_of(new), max_new=max(new), lse=True)
    assert nm.device_status() == nm.NM_OK
    at = 0
    for s, n in enumerate(new):
        rows = slice(at, at + n)
        want = definition(f64(q[rows]), K[s], V[s], [lens[s] - n + i + 1 for i in range(n)], 128 ** -0.5)
        compare(out[rows], lse[rows], want, lens[s], np.abs(V[s]).max())
        at += n
    o2, l2 = c.attention(0, q, starts=starts_of(new), max_new=max(new), lse=True)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_prompt_attention_past_4_gib(nm):
    """The prompt kernel on pages whose bytes lie past 2^32 of the pool."""
    P, L, Hk, D, H, n_new = 128, 32, 8, 128, 16, 70  # 1120 query rows
    per = nm.lib().nm_kv4_page_bytes(P, L, Hk, D)
    n = (1 << 32) // per + 8
    c = nm.Kv4Cache(n, P, L, Hk, D, 1, 4)
    c.refs.fill_(1)  # only the last three pages are free
    c.refs[n - 3:] = 0
    c.info[0] = 3
    c.reserve(starts=ints([0, 300]))
    assert int(c.tables[0, 0]) == n - 3 and (n - 3) * per > 1 << 32
    k, v = values(300, Hk, D, 41), values(300, Hk, D, 42)
    c.append(L - 1, k, v, starts=ints([0, 300]))
    rk, rv = ref.quantise(f32(k), f32(v))
    q = values(n_new, H, D, 43)
    out, lse = c.attention(L - 1, q, starts=ints([0, n_new]), max_new=n_new, lse=True)
    assert nm.device_status() == nm.NM_OK
    compare(out, lse, definition(f64(q), rk, rv, [300 - n_new + i + 1 for i in range(n_new)], D ** -0.5), 300,
            np.abs(rv).max())


# --- pages that are missing ----------------------------------------------------------------

@pytest.mark.parametrize("D,heads", [(128, 32), (64, 64)])
@pytest.mark.parametrize("max_new", [1, 64])
def test_attention_skips_tokens_of_missing_pages(nm, D, heads, max_new):
    """A token whose page the table does not name is not attended, by either kernel: it adds nothing to the
    sums, and a row that sees no other gives zeros."""
    lens, new, P = [300, 70], [40, 40], 32
    c, K, V = make(nm, lens, P=P, Hk=1, D=D, seed=101)
    q = values(80, heads, D, 102)
    for gone in ([4], [9], [0, 3, 8], list(range(9)), list(range(10))):
        saved = c.book.clone()
        for i, page in enumerate(gone):
            c.tables[0, page] = -1 if i % 2 else c.n_pages
        out, lse = c.attention(1, q, starts=starts_of(new), max_new=max_new, lse=True)
        assert nm.device_status() == nm.NM_ERR_BOUNDS
        c.book.copy_(saved)
        there = ~np.isin(np.arange(300) // P, gone)
        limits = [there & (np.arange(300) < 261 + i) for i in range(40)]
        compare(out[:40], lse[:40], definition(f64(q[:40]), K[0], V[0], limits, D ** -0.5), 300, np.abs(V[0]).max())
        want = definition(f64(q[40:]), K[1], V[1], [31 + i for i in range(40)], D ** -0.5)
        compare(out[40:], lse[40:], want, 70, np.abs(V[1]).max())
    assert nm.device_status() == nm.NM_OK


# --- rows that no sequence covers -------------------------------------------------------------

# starts, the tokens of the arrays, which rows have a sequence (its index), the status
COVERS = [
    ([0, 20, 30], 40, [(0, 20, 0), (20, 30, 1)], "NM_OK"),           # padding behind the last sequence
    ([3, 20, 40], 40, [(3, 20, 0), (20, 40, 1)], "NM_OK"),           # and before the first
    ([0, 20, 41], 40, [(0, 20, 0)], "NM_ERR_BOUNDS"),                # an end past the arrays
    ([-1, 20, 40], 40, [(20, 40, 1)], "NM_ERR_BOUNDS"),              # a start before them
    ([0, 30, 20], 40, [(0, 30, 0)], "NM_ERR_BOUNDS"),                # an end before its start
    ([0, 100, 200], 40, [], "NM_ERR_BOUNDS"),
    ([0, 0, 0], 40, [], "NM_OK"),
]


def attend_into(nm, c, layer, q, starts, max_new):
    """attention with out and lse full of NaN before the call."""
    T, H, D = q.shape
    out = torch.full((T, H * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), float("nan"), device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert nm.lib().nm_kv4_attention(c._ref, layer, None, starts.data_ptr(), starts.numel() - 1, T, max_new, q.data_ptr(),
                                     H * D, H, D ** -0.5, out.data_ptr(), H * D, lse.data_ptr(), s) == nm.NM_OK
    return out.view(T, H, D), lse


@pytest.mark.parametrize("D,heads,max_new", [(128, 2, 1), (64, 8, 8), (128, 64, 64), (64, 64, 64)])
@pytest.mark.parametrize("starts,T,rows,status", COVERS)
def test_attention_rows_of_no_sequence_are_zero(nm, D, heads, max_new, starts, T, rows, status):
    c, K, V = make(nm, [50, 90], Hk=2, D=D, seed=111)
    q = values(T, heads, D, 112)
    out, lse = attend_into(nm, c, 1, q, ints(starts), max_new)
    assert nm.device_status() == getattr(nm, status)
    none = np.ones(T, bool)
    for a, b, s in rows:
        none[a:b] = False
        n = b - a
        want = definition(f64(q[a:b]), K[s], V[s], [len(K[s]) - n + i + 1 for i in range(n)], D ** -0.5)
        compare(out[a:b], lse[a:b], want, len(K[s]), np.abs(V[s]).max())
    none = torch.from_numpy(none).cuda()
    assert bool((out[none] == 0).all()) and bool(torch.isneginf(lse[none]).all())


@pytest.mark.parametrize("heads,max_new", [(2, 1), (2, 9), (4, 1000)])
def test_attention_padding_behind_many_sequences(nm, heads, max_new):
    n, T = 700, 700 + 61
    lens = [1 + i % 37 for i in range(n)]
    c, K, V = make(nm, lens, P=16, L=1, Hk=1, D=64, seed=113)
    q = values(T, heads, 64, 114)
    out, lse = attend_into(nm, c, 0, q, ints(range(n + 1)), max_new)
    assert nm.device_status() == nm.NM_OK
    assert bool((out[n:] == 0).all()) and bool(torch.isneginf(lse[n:]).all())
    for s in (0, 1, 511, 512, 699):
        compare(out[s:s + 1], lse[s:s + 1], definition(f64(q[s:s + 1]), K[s], V[s], [lens[s]], 0.125), lens[s],
                np.abs(V[s]).max())


def read_into(nm, c, layer, T, starts, f32=True, k=True, v=True):
    """read with both results full of NaN before the call; None for one that is not asked for."""
    shape = (T, c.n_kv_heads, c.head_dim)
    res = [torch.full(shape, float("nan"), dtype=torch.float32 if f32 else torch.bfloat16, device="cuda") if x else None
           for x in (k, v)]
    s = torch.cuda.current_stream().cuda_stream
    assert nm.lib().nm_kv4_read(c._ref, layer, None, starts.data_ptr(), starts.numel() - 1, T,
                                *[None if x is None else x.data_ptr() for x in res], int(f32), s) == nm.NM_OK
    return res


@pytest.mark.parametrize("D,f32_", [(128, True), (128, False), (64, True), (64, False)])
@pytest.mark.parametrize("starts,T,rows,status", COVERS)
def test_read_rows_of_no_sequence_are_zero(nm, D, f32_, starts, T, rows, status):
    c, K, V = make(nm, [50, 90], Hk=3, D=D, seed=115)
    k, v = read_into(nm, c, 1, T, ints(starts), f32=f32_)
    assert nm.device_status() == getattr(nm, status)
    none = np.ones(T, bool)
    for a, b, s in rows:
        none[a:b] = False
        for got, held in ((k, K[s]), (v, V[s])):
            want = held[len(held) - (b - a):]
            np.testing.assert_array_equal(f32(got[a:b]), want if f32_ else ref.bf16(want))
    none = torch.from_numpy(none).cuda()
    assert bool((k[none] == 0).all()) and bool((v[none] == 0).all())
    only, _ = read_into(nm, c, 1, T, ints(starts), f32=f32_, v=False)
    assert torch.equal(only, k)
    nm.device_status()


@pytest.mark.parametrize("starts,T", [([-1, 1, 2], 2), ([-5, -5, 2], 2), ([0, 50, 3, 8], 60), ([0, 1, 1 << 30], 2),
                                      ([0, 2, 3], 2)])
def test_append_and_read_report_starts_out_of_range(nm, starts, T):
    c, _, _ = make(nm, [60] * (len(starts) - 1), seed=116)
    k = values(T, 2, 128, 117)
    c.append(1, k, k, starts=ints(starts))
    assert nm.device_status() == nm.NM_ERR_BOUNDS
    c.read(1, T, starts=ints(starts))
    assert nm.device_status() == nm.NM_ERR_BOUNDS
    good = [0] * (len(starts) - 1) + [T]
    c.append(1, k, k, starts=ints(good))
    c.read(1, T, starts=ints(good))
    assert nm.device_status() == nm.NM_OK


@pytest.mark.parametrize("D,heads,max_new", [(128, 2, 1), (64, 64, 64)])
def test_calls_with_tokens_and_no_sequence(nm, D, heads, max_new):
    """No sequence is listed: every row belongs to none."""
    T = 40
    c, _, _ = make(nm, [50, 90], Hk=2, D=D, seed=118)
    pool = c.pool.clone()
    q = values(T, heads, D, 119)
    out, lse = attend_into(nm, c, 1, q, ints([0]), max_new)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    k, v = read_into(nm, c, 1, T, ints([0]))
    assert bool((k == 0).all()) and bool((v == 0).all())
    k = values(T, 2, D, 120)
    qo = c.append(1, k, k, q=q, rope=rope_table(100, D), starts=ints([0]), q_out=torch.full_like(q, float("nan")))
    assert bool((qo == 0).all()) and torch.equal(c.pool, pool) and nm.device_status() == nm.NM_OK


# --- append ---------------------------------------------------------------------------------

@pytest.mark.parametrize("D,heads,T", [(128, 32, 8192), (64, 17, 16384), (128, 6, 50)])
def test_append_turns_q_in_place_as_it_does_beside(nm, D, heads, T):
    """q_out may be q itself, with many tokens (a warp turns several heads) and few."""
    c = nm.Kv4Cache(T // 128 + 1, 128, 1, 1, D, 1, T // 128 + 1)
    c.reserve(starts=ints([0, T]))
    k, q, rope = values(T, 1, D, 121), values(T, heads, D, 122), rope_table(T, D)
    beside = c.append(0, k, k, q=q, rope=rope, starts=ints([0, T]))
    c.append(0, k, k, q=q, rope=rope, starts=ints([0, T]), q_out=q)
    assert torch.equal(q, beside) and nm.device_status() == nm.NM_OK


def test_append_past_the_rope_table_and_again(nm):
    """Tokens past the rope table are not written and the status tells; appended again with a table that
    reaches them, the sequence is as if it had always been."""
    D, T = 128, 70
    c, K, V = make(nm, [30], P=64, Hk=1, seed=123, max_seqs=2)
    c.reserve(seqs=ints([1]), starts=ints([0, T]))
    k, v = values(T, 1, D, 124), values(T, 1, D, 125)
    rope = rope_table(T, D)
    c.append(1, k, v, rope=rope[:50].contiguous(), seqs=ints([1]), starts=ints([0, T]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS
    q = values(20, 64, D, 126)
    out, lse = c.attention(1, q, seqs=ints([0]), starts=ints([0, 20]), max_new=20, lse=True)
    compare(out, lse, definition(f64(q), K[0], V[0], [11 + i for i in range(20)], D ** -0.5), 30, np.abs(V[0]).max())
    c.append(1, k, v, rope=rope, seqs=ints([1]), starts=ints([0, T]))
    cs = rope.cpu().numpy()
    rk, rv = ref.quantise(ref.rotate(f32(k), cs[:, :64], cs[:, 64:]), f32(v))
    out, lse = c.attention(1, q, seqs=ints([1]), starts=ints([0, 20]), max_new=20, lse=True)
    compare(out, lse, definition(f64(q), rk, rv, [51 + i for i in range(20)], D ** -0.5), T, np.abs(rv).max())
    assert nm.device_status() == nm.NM_OK


@pytest.mark.parametrize("D", [128, 64])
def test_append_leaves_pages_that_are_shared(nm, D):
    """A reserve that finds no page refuses; an append all the same would fall on the sequence's last tokens,
    in a page that a fork reads. It is not written there, and the status tells."""
    P = 16
    c, K, V = make(nm, [32], P=P, Hk=2, D=D, extra=0, seed=141, max_seqs=3)
    c.fork(ints([0, 0]), ints([1, 2]))
    c.reserve(ints([0, 1]))
    assert c.info.tolist()[:2] == [0, 2] and c.lens.tolist() == [32, 32, 32]
    pool = c.pool.clone()
    k = values(2, 2, D, 142)
    c.append(1, k, k, seqs=ints([0, 1]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(c.pool, pool)
    c.append(1, values(5, 2, D, 143), values(5, 2, D, 144), seqs=ints([2]), starts=ints([0, 5]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(c.pool, pool)
    # with a page of its own a sequence is written as ever
    c.free(ints([1, 2]))
    c.append(1, k[:1], k[:1], seqs=ints([0]))
    kk, vv = c.read(1, 1, seqs=ints([0]), f32=True)
    rk, rv = ref.quantise(f32(k[:1]), f32(k[:1]))
    assert nm.device_status() == nm.NM_OK
    np.testing.assert_array_equal(f32(kk), rk)
    np.testing.assert_array_equal(f32(vv), rv)


# --- a second device ----------------------------------------------------------------------------

def test_attention_on_a_second_device(nm):
    """Both attention kernels on one device, then on another, in one process."""
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    results = []
    for d in (0, 1):
        torch.cuda.set_device(d)
        try:
            nm.init()
            c = nm.Kv4Cache(8, 32, 1, 1, 128, 1, 8, device=f"cuda:{d}")
            st = torch.tensor([0, 100], dtype=torch.int32, device=f"cuda:{d}")
            k, q = (values(100, h, 128, 131).cpu().to(f"cuda:{d}") for h in (1, 16))
            c.reserve(starts=st)
            c.append(0, k, k, starts=st)
            results.append([c.attention(0, q, starts=st, max_new=m).cpu() for m in (1, 100)])
            assert nm.device_status() == nm.NM_OK
        finally:
            torch.cuda.set_device(0)
    assert all(torch.equal(a, b) for a, b in zip(*results))
