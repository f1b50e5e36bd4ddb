"""The 4-bit paged KV cache against its references (oracle/kv4.py) on a GPU.

Tolerances, from the arithmetic:
* what append writes and read returns, and the rotated q: the format's fp32
  operations are fixed one by one, so the comparison is exact;
* scores: exact products, fp32 sums of D + 8 terms, so off by at most
  (D + 8) 2^-24 B < 2^-16 B, B = sum_d |q_d k_d| scale; log and exp add a few
  2^-22 of a base-2 exponent below 2^7: |lse - lse64| <= 2^-16 B + 2^-15;
* out: the weights and v are rounded to fp16 (2^-11 each), the weights carry the
  scores' error e (a factor e^2e), and the result is rounded to bf16 (2^-9):
  |out - out64| <= 2^-8 |out64| + (2^-10 + 2 e + 2^-14) A, A = sum_t weight |v_t|,
  plus, for weights below fp16's normal range, n 2^-30 max |v|.
"""
import numpy as np
import pytest
import torch

from oracle import kv4 as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    from sparse_decoding_gb300 import build
    build.build()
    import sparse_decoding_gb300 as nm
    torch.cuda.set_device(0)
    nm.init()
    return nm


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def starts_of(new):
    return ints(np.concatenate([[0], np.cumsum(new)]))


def rope_table(n, D):
    a = np.arange(n)[:, None] * (10000.0 ** (-np.arange(0, D, 2) / D))
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)).cuda()


def values(T, H, D, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, D, generator=g) * scale + torch.randn(1, H, D, generator=g) * scale).bfloat16().cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def f32(t):
    return t.float().cpu().numpy()


def make(nm, lens, P=32, L=2, Hk=2, D=128, extra=3, seed=0, garbage=True, max_seqs=None):
    """A cache whose sequences hold `lens` tokens of values(): (cache, K, V as held, fp32 per sequence)."""
    need = [-(-n // P) for n in lens]
    c = nm.Kv4Cache(sum(need) + extra, P, L, Hk, D, max_seqs or len(lens), max(need + [1]) + 1)
    if garbage:  # whatever was in the pool before: any bits, NaN parameters among them
        g = torch.Generator(device="cuda").manual_seed(seed + 99)
        c.pool.copy_(torch.randint(0, 256, c.pool.shape, generator=g, device="cuda", dtype=torch.uint8))
        c.pool[:, ::2] |= 0x7C
    T = sum(lens)
    k, v = values(T, Hk, D, seed), values(T, Hk, D, seed + 1)
    st = starts_of(lens)
    c.reserve(starts=st)
    c.append(L - 1, k, v, starts=st)
    kk, vv = c.read(L - 1, T, starts=st, f32=True)
    cut = np.cumsum(lens)[:-1]
    return c, np.split(f32(kk), cut), np.split(f32(vv), cut)


def check_attention(nm, c, K, V, lens, new, heads, layer, seed=5, qscale=1.0, max_new=None, scale=None, q=None):
    D = c.head_dim
    T = sum(new)
    q = values(T, heads, D, seed, qscale) if q is None else q
    out, lse = c.attention(layer, q, starts=starts_of(new), max_new=max_new, scale=scale, lse=True)
    assert nm.device_status() == nm.NM_OK
    sc = D ** -0.5 if scale is None else scale
    at = 0
    for s, n in enumerate(new):
        if n == 0:
            continue
        o, l, A, B = ref.attention(f64(q[at:at + n]), K[s].astype(np.float64), V[s].astype(np.float64), lens[s], sc)
        e = 2.0 ** -16 * B + 2.0 ** -15
        got, gl = f64(out[at:at + n]), lse[at:at + n].cpu().numpy().astype(np.float64)
        vmax = np.abs(V[s]).max() if V[s].size else 0.0
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + lens[s] * 2.0 ** -30 * vmax + 1e-30
        seen = np.isfinite(l)
        assert np.array_equal(np.isneginf(gl), np.isneginf(l)), "rows that see nothing"
        assert np.all(got[~seen & ~np.isnan(l)] == 0)
        assert np.array_equal(np.isnan(gl), np.isnan(l))
        off = np.abs(gl[seen] - l[seen])
        assert np.all(off <= e[seen]), f"lse off by {off.max()}"
        err = np.abs(got - o)[seen]
        assert np.all(err <= tol[seen]), f"out off by {(err / tol[seen]).max()} of its tolerance"
        at += n
    return out, lse


# --- append and read ---------------------------------------------------------------

@pytest.mark.parametrize("D,Hk,Hq,P", [(128, 8, 32, 64), (64, 2, 14, 16), (128, 1, 5, 128), (64, 8, 8, 32)])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([16, 17, 15], [16, 1, 15]), ([130, 5, 77], [30, 0, 77]), ([300], [300])])
def test_append_read_exact(nm, D, Hk, Hq, P, lens, new):
    T, n = sum(new), len(lens)
    c = nm.Kv4Cache(sum(-(-x // P) for x in lens) + 1, P, 2, Hk, D, n, 32)
    c.pool.fill_(0xFF)
    old = [a - b for a, b in zip(lens, new)]
    c.reserve(starts=starts_of(old))
    c.reserve(starts=starts_of(new))
    k, v, q = values(T, Hk, D, 1), values(T, Hk, D, 2), values(T, Hq, D, 3)
    rope = rope_table(max(lens), D)
    qo = c.append(1, k, v, q=q, rope=rope, starts=starts_of(new))
    kk, vv = c.read(1, T, starts=starts_of(new), f32=True)
    assert nm.device_status() == nm.NM_OK
    pos = np.concatenate([np.arange(a - b, a) for a, b in zip(lens, new)])
    cs = rope.cpu().numpy()[pos]
    kr = ref.rotate(f32(k), cs[:, :D // 2], cs[:, D // 2:])
    rk, rv = ref.quantise(kr, f32(v))
    np.testing.assert_array_equal(kk.cpu().numpy(), rk)
    np.testing.assert_array_equal(vv.cpu().numpy(), rv)
    np.testing.assert_array_equal(f32(qo), ref.bf16(ref.rotate(f32(q), cs[:, :D // 2], cs[:, D // 2:])))
    kb, vb = c.read(1, T, starts=starts_of(new))
    np.testing.assert_array_equal(f32(kb), ref.bf16(rk))
    np.testing.assert_array_equal(f32(vb), ref.bf16(rv))
    # the pool's bytes, from the layout
    pool, tab = c.pool.cpu().numpy(), c.tables.cpu().numpy()
    for i in sorted({0, T // 2, T - 1}):
        s = int(np.searchsorted(np.cumsum(new), i, side="right"))
        for h in sorted({0, Hk - 1}):
            dk, dv = ref.decode(pool, tab[s, pos[i] // P], 1, h, pos[i] % P, 2, Hk, P, D)
            np.testing.assert_array_equal(dk, rk[i, h])
            np.testing.assert_array_equal(dv, rv[i, h])
    # the other layer, and what lies past the sequences, are untouched
    layer0 = c.pool.view(c.n_pages, 2, -1)[:, 0]
    assert bool((layer0 == 0xFF).all())


def test_append_strides_and_in_place(nm):
    """k, v and q as slices of one fused row, q rotated in place; no rotation without a table."""
    D, Hk, Hq = 128, 2, 6
    row = values(9, Hq + 2 * Hk, D, 7).view(9, -1)
    q, k, v = row[:, :Hq * D], row[:, Hq * D:(Hq + Hk) * D], row[:, (Hq + Hk) * D:]
    c = nm.Kv4Cache(4, 16, 1, Hk, D, 1, 4)
    c.reserve(starts=ints([0, 9]))
    want = row.clone()
    qo = c.append(0, k, v, q=q, starts=ints([0, 9]))
    assert torch.equal(qo, want[:, :Hq * D])
    rope = rope_table(9, D)
    c.append(0, k, v, q=q, rope=rope, starts=ints([0, 9]), q_out=q)
    cs = rope.cpu().numpy()
    np.testing.assert_array_equal(f32(q).reshape(9, Hq, D),
                                  ref.bf16(ref.rotate(f32(want[:, :Hq * D]).reshape(9, Hq, D), cs[:, :64], cs[:, 64:])))
    assert torch.equal(k, want[:, Hq * D:(Hq + Hk) * D])
    kk, vv = c.read(0, 9, starts=ints([0, 9]), f32=True)
    rk, rv = ref.quantise(ref.rotate(f32(k).reshape(9, Hk, D), cs[:, :64], cs[:, 64:]), f32(v).reshape(9, Hk, D))
    np.testing.assert_array_equal(kk.cpu().numpy(), rk)
    np.testing.assert_array_equal(vv.cpu().numpy(), rv)


@pytest.mark.parametrize("D", [64, 128])
def test_append_edge_values(nm, D):
    """Equal channels, zeros, saturation, tiny and subnormal values, NaN and infinities."""
    T = 12
    k, v = values(T, 2, D, 11), values(T, 2, D, 12)
    k[0], v[0] = 0.0, -0.0
    k[1], v[1] = 3.25, -7.5
    k[2, :, 3], v[2, :, 5] = 1e6, -3e38
    k[3] *= 1e-4
    v[4] *= 1e-7
    v[5] *= 1e-38
    k[6, 0, 1] = float("nan")
    k[7, 1, 2] = float("inf")
    v[8, 0, D - 1] = float("nan")
    v[9, 1, 0] = float("-inf")
    k[10] = 32768.0
    k[10, :, 0] = -32768.0
    c = nm.Kv4Cache(2, 16, 1, 2, D, 1, 2)
    c.reserve(starts=ints([0, T]))
    c.append(0, k, v, starts=ints([0, T]))
    kk, vv = c.read(0, T, starts=ints([0, T]), f32=True)
    rk, rv = ref.quantise(f32(k), f32(v))
    np.testing.assert_array_equal(kk.cpu().numpy(), rk)
    np.testing.assert_array_equal(vv.cpu().numpy(), rv)
    assert np.isnan(rk[6, 0]).all() and np.isnan(rk[8, 0]).all() and np.isfinite(rk[6, 1]).all() and np.isfinite(rv).all()
    assert np.isfinite(rk[10]).all()


# --- attention -----------------------------------------------------------------------

CASES = [
    ([1], [1]), ([2], [1]), ([15], [1]), ([16], [1]), ([17], [1]), ([129], [1]), ([1000], [1]), ([4100], [1]),
    ([33, 1, 700, 64, 0, 16], [1, 1, 1, 1, 0, 1]),
    ([70, 35, 9], [3, 5, 9]), ([40, 300], [0, 13]),
]


@pytest.mark.parametrize("D,Hk,Hq,P", [(128, 2, 8, 64), (128, 2, 10, 32), (64, 2, 14, 16), (128, 1, 16, 128), (64, 3, 3, 32),
                                       (128, 1, 33, 16)])
@pytest.mark.parametrize("lens,new", CASES)
def test_attention(nm, D, Hk, Hq, P, lens, new):
    c, K, V = make(nm, lens, P=P, Hk=Hk, D=D, seed=sum(lens))
    check_attention(nm, c, K, V, lens, new, Hq, 1, max_new=max(new))


@pytest.mark.parametrize("D,Hk,Hq,P", [(128, 2, 8, 64), (128, 2, 10, 16), (64, 1, 7, 32), (128, 1, 1, 64), (64, 1, 64, 128)])
@pytest.mark.parametrize("lens,new", [([200], [200]), ([129, 64, 300], [129, 64, 100]), ([17, 0, 260, 140], [17, 0, 31, 140]),
                                      ([700], [33]), ([1200, 300], [1040, 30])])
def test_attention_prompts(nm, D, Hk, Hq, P, lens, new):
    c, K, V = make(nm, lens, P=P, Hk=Hk, D=D, seed=sum(lens) + 1)
    out, lse = check_attention(nm, c, K, V, lens, new, Hq, 1, max_new=max(new))
    # the bound only chooses the kernel
    few, lf = check_attention(nm, c, K, V, lens, new, Hq, 1, max_new=1)
    assert bool(torch.isclose(lse, lf, rtol=0, atol=1e-3).all())


@pytest.mark.parametrize("D,Hq", [(128, 1), (128, 4), (64, 7), (64, 1), (128, 64)])
@pytest.mark.parametrize("rows", [17, 23, 24, 25, 31, 33, 48, 49, 63, 64, 65, 72])
def test_attention_of_one_and_several_tiles(nm, D, Hq, rows):
    new = -(-rows // Hq)
    lens, news = [new + 5, 3001, 0, 64], [new, new, 0, 1]  # one sequence is cut over the CTAs
    c, K, V = make(nm, lens, P=16, L=1, Hk=1, D=D, seed=rows)
    check_attention(nm, c, K, V, lens, news, Hq, 0, max_new=new)
    lens, news = [80] * 200, [new] * 200  # more segments than CTAs
    c, K, V = make(nm, lens, P=16, L=1, Hk=1, D=D, seed=rows)
    check_attention(nm, c, K, V, lens, news, Hq, 0, max_new=new)


def test_attention_rows_with_nothing_to_attend(nm):
    """More new tokens than the sequence has, and an empty sequence: zeros and -inf."""
    lens, new = [5, 0, 20], [8, 3, 25]
    c, K, V = make(nm, lens, seed=3)
    out, lse = check_attention(nm, c, K, V, lens, new, 8, 1, max_new=25)
    assert bool((out[:3] == 0).all()) and bool(torch.isneginf(lse[:3]).all()) and bool(torch.isneginf(lse[8:11]).all())
    check_attention(nm, c, K, V, lens, new, 8, 1, max_new=1)
    check_attention(nm, c, K, V, lens, new, 64, 1, max_new=25)


@pytest.mark.parametrize("max_new,heads", [(1, 4), (64, 4), (64, 32)])
def test_attention_nonfinite_tokens_stay_where_they_are(nm, max_new, heads):
    """A token with NaN in k or v makes the queries that attend it NaN, and no others."""
    for D in (64, 128):
        lens = [90]
        k, v = values(90, 1, D, 21), values(90, 1, D, 22)
        k[70, 0, 3] = float("nan")
        v[80, 0, 5] = float("inf")
        for bad, first in ((k, 70), (v, 80)):
            kk, vv = (k, values(90, 1, D, 22)) if bad is k else (values(90, 1, D, 21), v)
            c = nm.Kv4Cache(6, 16, 1, 1, D, 1, 6)
            c.reserve(starts=ints([0, 90]))
            c.append(0, kk, vv, starts=ints([0, 90]))
            K, V = c.read(0, 90, starts=ints([0, 90]), f32=True)
            out, lse = check_attention(nm, c, [f32(K)], [f32(V)], lens, [40], heads, 0, max_new=max_new)
            at = first - 50
            assert bool(torch.isfinite(out[:at]).all()) and bool(torch.isnan(out[at:]).all())


@pytest.mark.parametrize("max_new,heads", [(1, 4), (64, 4), (64, 32)])
def test_attention_sharp_and_large_scores(nm, max_new, heads):
    """Scores far apart: one token takes all, or a first token with nearly no value takes the weight."""
    c, K, V = make(nm, [333], Hk=1, seed=8)
    for qs in (0.0, 1e-20, 30.0, 1e4):
        check_attention(nm, c, K, V, [333], [40], heads, 1, qscale=qs, max_new=max_new)
    check_attention(nm, c, K, V, [333], [40], heads, 1, qscale=1.0, scale=-0.7, max_new=max_new)
    check_attention(nm, c, K, V, [333], [40], heads, 1, qscale=1.0, scale=0.0, max_new=max_new)
    # a first token along q, with a small value
    D = 128
    k, v = values(333, 1, D, 31), values(333, 1, D, 32)
    q = torch.ones(40, heads, D, dtype=torch.bfloat16, device="cuda")
    k[0], v[0] = 1.4, 1e-3
    c = nm.Kv4Cache(12, 32, 1, 1, D, 1, 12)
    c.reserve(starts=ints([0, 333]))
    c.append(0, k, v, starts=ints([0, 333]))
    K, V = c.read(0, 333, starts=ints([0, 333]), f32=True)
    check_attention(nm, c, [f32(K)], [f32(V)], [333], [40], heads, 0, q=q, max_new=max_new)


def test_attention_strides_ids_and_streams(nm):
    """q and out as slices, listed sequences in another order, on a stream of its own."""
    lens = [40, 7, 90, 33]
    c, K, V = make(nm, lens, seed=13)
    wide = values(3, 8 + 5, 128, 14)
    q = wide[:, :8]
    order = [2, 0, 3]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        buf = torch.full((3, 20 * 128), 5.0, dtype=torch.bfloat16, device="cuda")
        out = buf[:, 128:9 * 128]
        c.attention(1, q, seqs=ints(order), out=out)
    torch.cuda.current_stream().wait_stream(s)
    assert bool((buf[:, :128] == 5).all()) and bool((buf[:, 9 * 128:] == 5).all())
    for i, sq in enumerate(order):
        o, _, A, B = ref.attention(f64(q[i:i + 1]), K[sq].astype(np.float64), V[sq].astype(np.float64), lens[sq], 128 ** -0.5)
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2.0 ** -13 + 2.0 ** -15 * B[..., None]) * A + 1e-6
        assert np.all(np.abs(f64(out[i]).reshape(1, 8, 128) - o) <= tol)


def test_attention_long_cut_over_many_ctas(nm):
    lens = [30011, 17, 9000]
    c, K, V = make(nm, lens, P=64, L=1, Hk=1, seed=17)
    out, lse = check_attention(nm, c, K, V, lens, [1, 1, 1], 8, 0, max_new=1)
    o2, l2 = c.attention(0, values(3, 8, 128, 5), lse=True)
    assert torch.equal(out, o2) and torch.equal(lse, l2), "results repeat bit for bit"
    check_attention(nm, c, K, V, lens, [7, 2, 5], 8, 0, max_new=7)
    check_attention(nm, c, K, V, lens, [20, 2, 5], 8, 0, max_new=20)


def test_attention_past_4_gib(nm):
    """Pages whose bytes lie past 2^32 of the pool."""
    P, L, Hk, D = 128, 32, 8, 128
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
    K, V = c.read(L - 1, 300, starts=ints([0, 300]), f32=True)
    rk, rv = ref.quantise(f32(k), f32(v))
    np.testing.assert_array_equal(K.cpu().numpy(), rk)
    np.testing.assert_array_equal(V.cpu().numpy(), rv)
    for new in (1, 40):
        check_attention(nm, c, [rk], [rv], [300], [new], 16, L - 1, max_new=new)


def test_graph_replays_follow_the_tables(nm):
    """A decode step captured once: reserve, append and attention, replayed as the sequences grow."""
    D, Hk, H = 128, 2, 8
    c, K, V = make(nm, [30, 5], P=16, L=1, Hk=Hk, extra=6, seed=51)
    K, V = [list(x) for x in K], [list(x) for x in V]
    k, v, q = (values(2, h, D, 52 + i) for i, h in enumerate((Hk, Hk, H)))
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        c.reserve(n=2)
        c.append(0, k, v)
        c.attention(0, q, out=out)
    for step in range(5):
        for i, t in enumerate((k, v, q)):
            t.copy_(values(2, t.shape[1], D, 60 + 3 * step + i))
        g.replay()
        rk, rv = ref.quantise(f32(k), f32(v))
        for s_ in range(2):
            K[s_].append(rk[s_])
            V[s_].append(rv[s_])
            o, _, A, B = ref.attention(f64(q[s_:s_ + 1]), np.array(K[s_], np.float64), np.array(V[s_], np.float64), len(K[s_]),
                                       D ** -0.5)
            tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2.0 ** -13 + 2.0 ** -15 * B[..., None]) * A + 1e-6
            assert np.all(np.abs(f64(out[s_:s_ + 1]) - o) <= tol)
    assert c.lens.tolist() == [35, 10] and nm.device_status() == nm.NM_OK


# --- pages -----------------------------------------------------------------------------

def same_book(c, m):
    assert c.lens.tolist() == m.lens
    assert c.refs.tolist() == m.refs
    assert c.tables.tolist() == m.tables
    assert c.info.tolist() == [len(m.free_pages()), m.result, m.moved] + [0] * 13


@pytest.mark.parametrize("seed", range(4))
def test_pages_random_walk(nm, seed):
    """Reserve, fork, free and compact in random order, refusals and shortage among them: tables equal the
    model's after every call, and pool bytes follow."""
    r = np.random.RandomState(seed)
    P = [16, 32, 64, 128][seed]
    n_pages, S, MP, L, Hk, D = [61, 40, 25, 23][seed], 9, 12, 2, 2, 64
    c = nm.Kv4Cache(n_pages, P, L, Hk, D, S, MP)
    c.pool.copy_(torch.from_numpy(r.randint(0, 256, c.pool.shape).astype(np.uint8)))
    m = ref.Pages(n_pages, P, S, MP)
    pool = c.pool.cpu().numpy().copy()
    cell = 16 * (D + 8 * (D // 64))
    for _ in range(40):
        what = r.randint(4)
        ids = r.permutation(S)[:r.randint(1, 5)].tolist()
        if what == 0:
            new = [int(r.randint(0, 3 * P)) for _ in ids]
            if r.rand() < 0.15:
                ids[-1] = ids[0] if r.rand() < 0.5 else S
            c.reserve(ints(ids), starts_of(new))
            m.reserve(ids, new)
        elif what == 1:
            src = [int(r.randint(S)) for _ in ids]
            empty = [i for i in range(S) if m.lens[i] == 0]
            dst = empty[:len(src)] if r.rand() < 0.8 else ids
            src = src[:len(dst)]
            c.fork(ints(src), ints(dst))
            m.fork(src, dst)
            v = pool.reshape(n_pages, L * Hk, P // 16, cell)
            for a, b, tokens in (m.copies if m.result == 0 else []):
                v[b, :, :-(-tokens // 16)] = v[a, :, :-(-tokens // 16)]
        elif what == 2:
            ids = ids + ids[:1]  # twice is once
            c.free(ints(ids))
            m.free(ids)
        else:
            c.compact()
            m.compact()
            for a, b in m.copies:
                pool[b] = pool[a]
        same_book(c, m)
        assert np.array_equal(c.pool.cpu().numpy(), pool)
    assert nm.device_status() == nm.NM_OK


def test_pages_many_sequences_and_large_pool(nm):
    """1024 sequences in a call; a pool whose free pages lie far apart."""
    n_pages, P, S, MP = 9001, 16, 1024, 12
    c = nm.Kv4Cache(n_pages, P, 1, 1, 64, S, MP)
    m = ref.Pages(n_pages, P, S, MP)
    r = np.random.RandomState(0)
    new = r.randint(0, 8 * P, S).tolist()
    c.reserve(starts=starts_of(new))
    m.reserve(list(range(S)), new)
    same_book(c, m)
    gone = r.permutation(S)[:600].tolist()
    c.free(ints(gone))
    m.free(gone)
    same_book(c, m)
    src, dst = [i for i in range(S) if m.lens[i]][:200], gone[:200]
    c.fork(ints(src), ints(dst))
    m.fork(src, dst)
    same_book(c, m)
    c.compact()
    m.compact()
    same_book(c, m)
    c.reserve(ints(list(range(S))), starts_of([1] * S))
    m.reserve(list(range(S)), [1] * S)
    same_book(c, m)


def test_fork_shares_and_attends(nm):
    """Forked sequences read the parent's tokens and write only their own pages; after the parent is freed
    and the pool compacted they still hold them."""
    D, Hk, P = 128, 2, 16
    c, K, V = make(nm, [45], P=P, L=2, Hk=Hk, extra=8, seed=71, max_seqs=3)
    c.fork(ints([0, 0]), ints([1, 2]))
    c.reserve(ints([0, 1, 2]))
    k, v = values(3, Hk, D, 72), values(3, Hk, D, 73)
    c.append(1, k, v, seqs=ints([0, 1, 2]))
    rk, rv = ref.quantise(f32(k), f32(v))
    c.free(ints([0]))
    c.compact()
    assert c.info.tolist()[:3] == [c.n_pages - 4, 0, 1]
    q = values(2, 8, D, 74)
    out = c.attention(1, q, seqs=ints([1, 2]))
    for i in (0, 1):
        kk = np.concatenate([K[0], rk[i + 1:i + 2]]).astype(np.float64)
        vv = np.concatenate([V[0], rv[i + 1:i + 2]]).astype(np.float64)
        o, _, A, B = ref.attention(f64(q[i:i + 1]), kk, vv, 46, D ** -0.5)
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2.0 ** -13 + 2.0 ** -15 * B[..., None]) * A + 1e-6
        assert np.all(np.abs(f64(out[i:i + 1]) - o) <= tol)


def test_copy_pages(nm):
    a = nm.Kv4Cache(7, 32, 3, 2, 64, 1, 4)
    b = nm.Kv4Cache(5, 32, 3, 2, 64, 1, 4)
    r = np.random.RandomState(1)
    pa, pb = (r.randint(0, 256, x.pool.shape).astype(np.uint8) for x in (a, b))
    a.pool.copy_(torch.from_numpy(pa))
    b.pool.copy_(torch.from_numpy(pb))
    a.copy_pages(ints([6, 0, 3]), ints([1, 4, 0]), b)
    pb[[1, 4, 0]] = pa[[6, 0, 3]]
    assert np.array_equal(b.pool.cpu().numpy(), pb)
    a.copy_pages(ints([2, 5]), ints([4, 1]))
    pa[[4, 1]] = pa[[2, 5]]
    assert np.array_equal(a.pool.cpu().numpy(), pa)
    a.copy_pages(ints([7, 2]), ints([0, -1]))  # out of range: skipped, reported
    assert np.array_equal(a.pool.cpu().numpy(), pa) and nm.device_status() == nm.NM_ERR_BOUNDS
    assert nm.device_status() == nm.NM_OK


# --- tables that name nothing ------------------------------------------------------------

def test_tables_out_of_range_are_reported(nm):
    """Ids, lengths and pages out of range: nothing is followed, the status tells, other sequences are right."""
    D, Hk = 128, 2
    c, K, V = make(nm, [40, 40], seed=81)
    q = values(2, 8, D, 82)
    good = c.attention(1, q)
    assert nm.device_status() == nm.NM_OK
    bad = c.attention(1, q, seqs=ints([0, 2]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS
    assert torch.equal(bad[0], good[0]) and bool((bad[1] == 0).all())
    saved = c.book.clone()
    c.lens[1] = 1 << 29
    bad = c.attention(1, q)
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(bad[0], good[0]) and bool((bad[1] == 0).all())
    c.book.copy_(saved)
    c.tables[1, 0], c.tables[1, 1] = c.n_pages, -7
    pool = c.pool.clone()
    bad = c.attention(1, q)
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(bad[0], good[0])
    k = values(2, Hk, D, 83)
    c.append(1, k, k, seqs=ints([1, 5]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(c.pool, pool)
    kk, _ = c.read(1, 2, seqs=ints([1, 0]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and bool((kk[0] == 0).all())
    c.book.copy_(saved)
    # a rope table that ends before the position
    qo = c.append(1, k, k, q=q, rope=rope_table(39, D))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(c.pool, pool) and bool((qo == 0).all())
    # starts past the tokens: those sequences have none
    out = c.attention(1, q, starts=ints([0, 1, 3]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(out[0], good[0])
    assert torch.equal(c.attention(1, q), good) and nm.device_status() == nm.NM_OK


def test_read_rows_that_are_not_there(nm):
    """More rows asked for than a sequence has: zeros, and the status tells."""
    c, K, V = make(nm, [5, 0, 20], seed=91)
    k, v = c.read(1, 8 + 3 + 4, starts=starts_of([8, 3, 4]), f32=True)
    assert nm.device_status() == nm.NM_ERR_BOUNDS
    assert bool((k[:3] == 0).all()) and bool((v[:3] == 0).all()) and bool((k[8:11] == 0).all())
    np.testing.assert_array_equal(f32(k[3:8]), K[0])
    np.testing.assert_array_equal(f32(v[11:]), V[2][-4:])


@pytest.mark.parametrize("max_new,heads", [(1, 8), (64, 8), (64, 64)])
def test_attention_nonfinite_queries_stay_in_their_rows(nm, max_new, heads):
    c, K, V = make(nm, [100], seed=92)
    q = values(40, heads, 128, 93)
    good = c.attention(1, q, starts=ints([0, 40]), max_new=max_new)
    bad = q.clone()
    bad[7, 3, 11], bad[20, 6, 5] = float("nan"), float("inf")
    out = c.attention(1, bad, starts=ints([0, 40]), max_new=max_new)
    same = torch.ones(40, heads, dtype=torch.bool, device="cuda")
    same[7, 3] = same[20, 6] = False
    assert torch.equal(out[same], good[same]) and bool(torch.isnan(out[7, 3]).all())


@pytest.mark.parametrize("new,max_new", [(1, 1), (9, 9), (3, 1000)])
def test_attention_many_sequences(nm, new, max_new):
    """1024 sequences in a call, short ones and a long one, through each kernel."""
    n = 1024
    r = np.random.RandomState(new)
    lens = (r.randint(0, 40, n) + new).tolist()
    lens[700] = 3000
    c, K, V = make(nm, lens, P=16, L=1, Hk=1, D=64, seed=94)
    q = values(n * new, 4, 64, 95)
    out, lse = c.attention(0, q, starts=starts_of([new] * n), max_new=max_new, lse=True)
    assert nm.device_status() == nm.NM_OK
    for s in (0, 1, 511, 512, 513, 699, 700, 701, 1023):
        rows = slice(s * new, (s + 1) * new)
        o, l, A, B = ref.attention(f64(q[rows]), K[s].astype(np.float64), V[s].astype(np.float64), lens[s], 0.125)
        e = 2.0 ** -16 * B + 2.0 ** -15
        assert np.all(np.abs(f64(lse[rows]) - l) <= e)
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + lens[s] * 2.0 ** -30 * 8
        assert np.all(np.abs(f64(out[rows]) - o) <= tol)


# --- used together -----------------------------------------------------------------------

def test_example_decode_loop(nm):
    """The example's loop: every attention result against the definition, on the q, k, v that went in."""
    from examples import paged_decode as ex
    d = ex.Decoder(layers=2, hidden=256, heads=8, kv_heads=2, dim=64, ffn=512, sequences=3, tokens=80, page=16, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    prompt = torch.randn(37, 256, generator=g, device="cuda").bfloat16()
    traces, step = [], d.step

    def traced(x, seqs, starts=None):
        t = []
        y = step(x, seqs, starts, trace=t)
        traces.append((seqs.tolist(), None if starts is None else starts.tolist(), t))
        return y

    d.step = traced
    out = ex.run(d, prompt, 3, 4)
    assert len(out) == 4 and nm.device_status() == nm.NM_OK
    rope = d.rope.cpu().numpy()
    held = [[([], []) for _ in range(2)] for _ in range(3)]  # [sequence][layer]: K, V as held
    for seqs, starts, layers in traces:
        if starts is None and len(held[1][0][0]) == 0:  # the fork came before the first joint step
            for s in (1, 2):
                held[s] = [(list(k), list(v)) for k, v in held[0]]
        starts = starts or list(range(len(seqs) + 1))
        for layer, (q, k, v, a) in enumerate(layers):
            q, k, v = (f32(t).reshape(t.shape[0], -1, 64) for t in (q, k, v))
            for i, s in enumerate(seqs):
                K, V = held[s][layer]
                rows = slice(starts[i], starts[i + 1])
                pos = np.arange(len(K), len(K) + starts[i + 1] - starts[i])
                cos, sin = rope[pos, :32], rope[pos, 32:]
                rk, rv = ref.quantise(ref.rotate(k[rows], cos, sin), v[rows])
                K.extend(rk)
                V.extend(rv)
                rq = ref.bf16(ref.rotate(q[rows], cos, sin)).astype(np.float64)
                o, _, A, B = ref.attention(rq, np.array(K, np.float64), np.array(V, np.float64), len(K), 0.125)
                e = 2.0 ** -16 * B[..., None] + 2.0 ** -15
                tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e + 2.0 ** -14) * A + 1e-6
                assert np.all(np.abs(f64(a[rows]).reshape(o.shape) - o) <= tol)
    assert d.cache.lens.tolist() == [41, 0, 0] and d.cache.info.tolist()[:2] == [d.cache.n_pages - 3, 0]
    assert d.cache.tables[0, :3].sort().values.tolist() == [0, 1, 2]
