"""The 8-bit paged KV cache against its references (oracle/kv8.py) on a GPU.

Tolerances, from the arithmetic:
* what append writes and read returns, bounds, lists of pages, and the rotated q: the format's
  operations are fixed one by one, so the comparison is exact;
* scores: exact products, fp32 sums of D terms and one product with a power of two, so off by at most
  (D + 2) 2^-24 B < 2^-16 B, B = sum_d |q_d k_d| scale; log and exp add a few 2^-22 of a
  base-2 exponent below 2^8: |lse - lse64| <= 2^-16 B + 2^-15;
* out: v is exact, the weights are rounded to fp16 (2^-11) and carry the scores' error e (a factor
  e^2e), and the result is rounded to bf16 (2^-9 .. 2^-8):
  |out - out64| <= 2^-8 |out64| + (2^-10 + 2 e + 2^-14) A, A = sum_t weight |v_t|,
  plus, for weights below fp16's normal range (2^-25 of codes up to 448 under a weight of at least 2^6, where
  448 of the heaviest block's scale is at most twice its largest |v|), n 2^-30 max |v|, or n 2^-46
  where the scale is the least there is.
"""
import numpy as np
import pytest
import torch

from oracle import kv4 as ref4
from oracle import kv8 as ref
from tests.test_gpu_kv4 import f32, f64, ints, rope_table, same_book, starts_of, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nm():
    from sparse_decoding_gb300 import build
    build.build()
    import sparse_decoding_gb300 as nm
    torch.cuda.set_device(0)
    nm.init()
    return nm


def drifting(T, H, D, seed, page):
    """Keys of which neighbours are alike, with a few large channels: pages differ."""
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(T, H, D, generator=g) + 1.5 * torch.randn(-(-T // page), H, D, generator=g).repeat_interleave(page, 0)[:T]
    k[:, :, ::29] *= 5.0
    return k.bfloat16().cuda()


def make(nm, lens, P=32, L=2, Hk=2, D=128, extra=3, seed=0, max_seqs=None):
    """A cache whose sequences hold `lens` tokens: (cache, ref.Sequence of each)."""
    need = [-(-n // P) for n in lens]
    c = nm.Kv8Cache(sum(need) + extra, P, L, Hk, D, max_seqs or len(lens), max(need + [1]) + 1)
    g = torch.Generator(device="cuda").manual_seed(seed + 99)
    c.pool.copy_(torch.randint(0, 256, c.pool.shape, generator=g, device="cuda", dtype=torch.uint8))
    c.pool[:, ::2] |= 0x7F  # whatever was in the pool before: NaN codes, NaN scales
    T = sum(lens)
    k, v = drifting(T, Hk, D, seed, P), values(T, Hk, D, seed + 1)
    st = starts_of(lens)
    c.reserve(starts=st)
    c.append(L - 1, k, v, starts=st)
    held = []
    for a, b in zip(np.cumsum([0] + lens), np.cumsum(lens)):
        held.append(ref.Sequence(Hk, D))
        held[-1].append(f32(k[a:b]), f32(v[a:b]))
    return c, held


def check(nm, c, held, new, heads, layer, seed=5, qscale=1.0, max_new=None, scale=None, q=None, pages=None):
    """One attention call against the definition; pages: None, or the lists on the device."""
    D = c.head_dim
    q = values(sum(new), heads, D, seed, qscale) if q is None else q
    out, lse = c.attention(layer, q, starts=starts_of(new), max_new=max_new, scale=scale, lse=True, pages=pages)
    assert nm.device_status() == nm.NM_OK
    sc = D ** -0.5 if scale is None else scale
    at = 0
    for s, n in enumerate(new):
        if n == 0:
            continue
        K, V = held[s].k.astype(np.float64), held[s].v.astype(np.float64)
        lists = None if pages is None else pages[at:at + n].cpu().numpy()
        o, l, A, B = ref.attention(f64(q[at:at + n]), K, V, len(K), sc, lists, c.page_tokens)
        e = 2.0 ** -16 * B + 2.0 ** -15
        got, gl = f64(out[at:at + n]), lse[at:at + n].cpu().numpy().astype(np.float64)
        vmax = np.abs(V).max() if V.size else 0.0
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + len(K) * (2.0 ** -30 * vmax + 2.0 ** -46)
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

@pytest.mark.parametrize("D,Hk,Hq,P", [(128, 8, 32, 64), (64, 2, 14, 16), (128, 1, 5, 128), (64, 3, 3, 32)])
@pytest.mark.parametrize("calls", [[[1]], [[16, 1, 15], [16, 16, 0]], [[100, 5, 0], [30, 0, 77]], [[300]], [[128], [1], [127]],
                                   [[3, 20]] + [[1, 1]] * 40])
def test_append_read_exact(nm, D, Hk, Hq, P, calls):
    """Tokens in several calls: codes, scales, values, bounds and the rotated q, bit for bit."""
    n = len(calls[0])
    lens = np.sum(calls, 0)
    c = nm.Kv8Cache(int(sum(-(-x // P) for x in lens)) + 1, P, 2, Hk, D, n, 32)
    c.pool.fill_(0xFF)
    rope = rope_table(int(max(lens)), D)
    cs = rope.cpu().numpy()
    held = [ref.Sequence(Hk, D) for _ in range(n)]
    for i, new in enumerate(calls):
        T = sum(new)
        # magnitudes that grow and shrink from call to call, so that scales have to move
        k, v, q = values(T, Hk, D, 7 * i + 1, 3.0 ** (i % 4)), values(T, Hk, D, 7 * i + 2, 2.0 ** (i % 9 - 4)), values(T, Hq, D, 3)
        c.reserve(starts=starts_of(new))
        qo = c.append(1, k, v, q=q, rope=rope, starts=starts_of(new))
        at = 0
        for s, m in enumerate(new):
            pos = np.arange(len(held[s].k), len(held[s].k) + m)
            cos, sin = cs[pos, :D // 2], cs[pos, D // 2:]
            held[s].append(ref.rotate(f32(k[at:at + m]), cos, sin), f32(v[at:at + m]))
            np.testing.assert_array_equal(f32(qo[at:at + m]), ref.bf16(ref.rotate(f32(q[at:at + m]), cos, sin)))
            at += m
    assert nm.device_status() == nm.NM_OK
    for dt in (True, False):
        kk, vv = c.read(1, int(sum(lens)), starts=starts_of(lens), f32=dt)
        np.testing.assert_array_equal(f32(kk), np.concatenate([h.k for h in held]))
        np.testing.assert_array_equal(f32(vv), np.concatenate([h.v for h in held]))
    # the pool's bytes, from the layout
    pool, tab = c.pool.cpu().numpy(), c.tables.cpu().numpy()
    for s in range(n):
        for pos in sorted({0, int(lens[s]) // 2, int(lens[s]) - 1} & set(range(int(lens[s])))):
            for h in sorted({0, Hk - 1}):
                (dk, dv), _ = ref.decode(pool, tab[s, pos // P], 1, h, pos % P, 2, Hk, P, D)
                np.testing.assert_array_equal(dk, held[s].k[pos, h])
                np.testing.assert_array_equal(dv, held[s].v[pos, h])
        for z in range(int(lens[s]) // P):
            up, low, step = ref.bounds(held[s].k[z * P:(z + 1) * P])
            for h in sorted({0, Hk - 1}):
                _, (u, w, st) = ref.decode(pool, tab[s, z], 1, h, 0, 2, Hk, P, D)
                np.testing.assert_array_equal(u, up[h])
                np.testing.assert_array_equal(w, low[h])
                assert st == step[h]
    # the other layer is untouched
    assert bool((c.pool.view(c.n_pages, 2, -1)[:, 0] == 0xFF).all())


def test_append_strides_and_in_place(nm):
    """k, v and q as slices of one fused row, q rotated in place; no rotation without a table."""
    D, Hk, Hq = 128, 2, 6
    row = values(9, Hq + 2 * Hk, D, 7).view(9, -1)
    q, k, v = row[:, :Hq * D], row[:, Hq * D:(Hq + Hk) * D], row[:, (Hq + Hk) * D:]
    c = nm.Kv8Cache(4, 16, 1, Hk, D, 1, 4)
    c.reserve(starts=ints([0, 9]))
    want = row.clone()
    assert torch.equal(c.append(0, k, v, q=q, starts=ints([0, 9])), want[:, :Hq * D])
    rope = rope_table(9, D)
    c.append(0, k, v, q=q, rope=rope, starts=ints([0, 9]), q_out=q)
    cs = rope.cpu().numpy()
    np.testing.assert_array_equal(f32(q).reshape(9, Hq, D),
                                  ref.bf16(ref.rotate(f32(want[:, :Hq * D]).reshape(9, Hq, D), cs[:, :64], cs[:, 64:])))
    kk, vv = c.read(0, 9, starts=ints([0, 9]), f32=True)
    h = ref.Sequence(Hk, D)
    h.append(ref.rotate(f32(k).reshape(9, Hk, D), cs[:, :64], cs[:, 64:]), f32(v).reshape(9, Hk, D))
    np.testing.assert_array_equal(f32(kk), h.k)
    np.testing.assert_array_equal(f32(vv), h.v)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("step", [1, 5, 40])
def test_append_edge_values(nm, D, step):
    """Zeros, saturation, tiny and subnormal values, code borders, NaN and infinities, in calls of 1, 5 or all tokens."""
    T = 40
    k, v = values(T, 2, D, 11), values(T, 2, D, 12)
    k[0], v[0] = 0.0, -0.0
    k[1], v[1] = 448.0, -224.0
    k[2, :, 3], v[2, :, 5] = 1e6, -3e38
    k[3] *= 1e-4
    v[4] *= 1e-9
    v[5] *= 1e-38
    k[6, 0, 1] = float("nan")
    k[7, 1, 2] = float("inf")
    v[8, 0, D - 1] = float("nan")
    v[9, 1, 0] = float("-inf")
    k[16:20], v[16:20] = 1e-7, 1e-20
    k[20:24] = torch.linspace(-480, 480, D).bfloat16().cuda()  # above and below the largest code
    k[24], v[24] = 32768.0, 1.0
    k[32:36], v[32:36] = 2.0 ** -9 * 1.5, 2.0 ** -10  # ties between the least codes
    v[36] = 448.0
    k[37, :, 0] = 449.0
    c = nm.Kv8Cache(3, 16, 1, 2, D, 1, 3)
    h = ref.Sequence(2, D)
    for a in range(0, T, step):
        b = min(T, a + step)
        c.reserve(starts=ints([0, b - a]))
        c.append(0, k[a:b], v[a:b], starts=ints([0, b - a]))
        h.append(f32(k[a:b]), f32(v[a:b]))
    kk, vv = c.read(0, T, starts=ints([0, T]), f32=True)
    np.testing.assert_array_equal(f32(kk), h.k)
    np.testing.assert_array_equal(f32(vv), h.v)
    assert np.isnan(h.k[6, 0]).all() and np.isnan(h.k[8, 0]).all() and np.isfinite(h.k[6, 1]).all() and np.isfinite(h.v).all()
    pool = c.pool.cpu().numpy()
    for z in (0, 1):
        up, low, stp = ref.bounds(h.k[16 * z:16 * z + 16])
        for head in (0, 1):
            _, (u, w, s) = ref.decode(pool, c.tables[0, z].item(), 0, head, 0, 1, 2, 16, D)
            np.testing.assert_array_equal(u, up[head])
            np.testing.assert_array_equal(w, low[head])
            assert s == stp[head]


# --- attention -----------------------------------------------------------------------

@pytest.mark.parametrize("D,Hk,Hq,P", [(128, 2, 8, 64), (128, 2, 10, 32), (64, 2, 14, 16), (128, 1, 16, 128), (64, 3, 3, 32),
                                       (128, 1, 33, 16)])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([2], [1]), ([15], [1]), ([16], [1]), ([17], [1]), ([129], [1]), ([1000], [1]),
                                      ([4100], [1]), ([33, 1, 700, 64, 0, 16], [1, 1, 1, 1, 0, 1]), ([70, 35, 9], [3, 5, 9]),
                                      ([40, 300], [0, 13])])
def test_attention(nm, D, Hk, Hq, P, lens, new):
    c, held = make(nm, lens, P=P, Hk=Hk, D=D, seed=sum(lens))
    check(nm, c, held, new, Hq, 1, max_new=max(new))


@pytest.mark.parametrize("D,Hk,Hq,P", [(128, 2, 8, 64), (128, 2, 10, 16), (64, 1, 7, 32), (128, 1, 1, 64), (64, 1, 64, 128)])
@pytest.mark.parametrize("lens,new", [([200], [200]), ([129, 64, 300], [129, 64, 100]), ([17, 0, 260, 140], [17, 0, 31, 140]),
                                      ([700], [33]), ([1200, 300], [1040, 30])])
def test_attention_prompts(nm, D, Hk, Hq, P, lens, new):
    c, held = make(nm, lens, P=P, Hk=Hk, D=D, seed=sum(lens) + 1)
    out, lse = check(nm, c, held, new, Hq, 1, max_new=max(new))
    # the bound only chooses the kernel
    few, lf = check(nm, c, held, new, Hq, 1, max_new=1)
    assert bool(torch.isclose(lse, lf, rtol=0, atol=1e-3).all())


@pytest.mark.parametrize("D,Hq", [(128, 1), (128, 4), (64, 7), (128, 64)])
@pytest.mark.parametrize("rows", [17, 24, 25, 33, 48, 49, 64, 65])
def test_attention_of_one_and_several_tiles(nm, D, Hq, rows):
    new = -(-rows // Hq)
    c, held = make(nm, [new + 5, 3001, 0, 64], P=16, L=1, Hk=1, D=D, seed=rows)  # one sequence is cut over the CTAs
    check(nm, c, held, [new, new, 0, 1], Hq, 0, max_new=new)
    c, held = make(nm, [80] * 200, P=16, L=1, Hk=1, D=D, seed=rows)  # more segments than CTAs
    check(nm, c, held, [new] * 200, Hq, 0, max_new=new)


@pytest.mark.parametrize("max_new,heads", [(1, 8), (25, 64)])
def test_attention_rows_with_nothing_to_attend(nm, max_new, heads):
    """More new tokens than the sequence has, and an empty sequence: zeros and -inf."""
    c, held = make(nm, [5, 0, 20], seed=3)
    out, lse = check(nm, c, held, [8, 3, 25], heads, 1, max_new=max_new)
    assert bool((out[:3] == 0).all()) and bool(torch.isneginf(lse[:3]).all()) and bool(torch.isneginf(lse[8:11]).all())


@pytest.mark.parametrize("max_new,heads", [(1, 4), (64, 32)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_nonfinite_tokens_stay_where_they_are(nm, max_new, heads, D):
    """A token with NaN in k or v makes the queries that attend it NaN, and no others."""
    for which, first in (("k", 70), ("v", 80)):
        k, v = values(90, 1, D, 21), values(90, 1, D, 22)
        if which == "k":
            k[70, 0, 3] = float("nan")
        else:
            v[80, 0, 5] = float("inf")
        c = nm.Kv8Cache(6, 16, 1, 1, D, 1, 6)
        c.reserve(starts=ints([0, 90]))
        c.append(0, k, v, starts=ints([0, 90]))
        h = ref.Sequence(1, D)
        h.append(f32(k), f32(v))
        out, lse = check(nm, c, [h], [40], heads, 0, max_new=max_new)
        assert bool(torch.isfinite(out[:first - 50]).all()) and bool(torch.isnan(out[first - 50:]).all())


@pytest.mark.parametrize("max_new,heads", [(1, 4), (64, 4), (64, 32)])
def test_attention_sharp_and_large_scores(nm, max_new, heads):
    """Scores far apart; blocks whose scales lie far apart, in K and in V."""
    c, held = make(nm, [333], Hk=1, seed=8)
    for qs in (0.0, 1e-20, 30.0, 1e4):
        check(nm, c, held, [40], heads, 1, qscale=qs, max_new=max_new)
    check(nm, c, held, [40], heads, 1, scale=-0.7, max_new=max_new)
    check(nm, c, held, [40], heads, 1, scale=0.0, max_new=max_new)
    D = 128
    k, v = values(333, 1, D, 31), values(333, 1, D, 32)
    for b, (x, y) in enumerate([(1e-6, 1.0), (1.0, 1e-6), (30.0, 3e4), (1.0, 1e-9), (1e-3, 1e3)] * 4):
        k[16 * b:16 * b + 16] *= x
        v[16 * b:16 * b + 16] *= y
    k[0], v[0] = 1.4, 1e-3
    c = nm.Kv8Cache(12, 32, 1, 1, D, 1, 12)
    c.reserve(starts=ints([0, 333]))
    c.append(0, k, v, starts=ints([0, 333]))
    h = ref.Sequence(1, D)
    h.append(f32(k), f32(v))
    check(nm, c, [h], [40], heads, 0, max_new=max_new)
    check(nm, c, [h], [40], heads, 0, max_new=max_new, q=torch.ones(40, heads, D, dtype=torch.bfloat16, device="cuda"))


def test_attention_strides_ids_and_streams(nm):
    """q and out as slices, listed sequences in another order, on a stream of its own."""
    lens = [40, 7, 90, 33]
    c, held = make(nm, lens, seed=13)
    q = values(3, 8 + 5, 128, 14)[:, :8]
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
        o, _, A, B = ref.attention(f64(q[i:i + 1]), held[sq].k.astype(np.float64), held[sq].v.astype(np.float64), lens[sq], 128 ** -0.5)
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2.0 ** -13 + 2.0 ** -15 * B[..., None]) * A + 1e-6
        assert np.all(np.abs(f64(out[i]).reshape(1, 8, 128) - o) <= tol)


def test_attention_long_cut_over_many_ctas(nm):
    c, held = make(nm, [30011, 17, 9000], P=64, L=1, Hk=1, seed=17)
    out, lse = check(nm, c, held, [1, 1, 1], 8, 0, max_new=1)
    o2, l2 = c.attention(0, values(3, 8, 128, 5), lse=True)
    assert torch.equal(out, o2) and torch.equal(lse, l2), "results repeat bit for bit"
    check(nm, c, held, [7, 2, 5], 8, 0, max_new=7)
    check(nm, c, held, [20, 2, 5], 8, 0, max_new=20)
    out, lse = check(nm, c, held, [150, 0, 3], 8, 0)
    o2, l2 = c.attention(0, values(153, 8, 128, 5), starts=starts_of([150, 0, 3]), lse=True)
    assert torch.equal(out, o2) and torch.equal(lse, l2), "results repeat bit for bit"


def test_attention_past_4_gib(nm):
    """Pages whose bytes lie past 2^32 of the pool, through every call."""
    P, L, Hk, D = 128, 32, 8, 128
    per = nm.lib().nm_kv8_page_bytes(P, L, Hk, D)
    n = (1 << 32) // per + 8
    c = nm.Kv8Cache(n, P, L, Hk, D, 1, 4)
    c.refs.fill_(1)  # only the last four pages are free
    c.refs[n - 4:] = 0
    c.info[0] = 4
    c.reserve(starts=ints([0, 400]))
    assert int(c.tables[0, 0]) == n - 4 and (n - 4) * per > 1 << 32
    k, v = values(400, Hk, D, 41), values(400, Hk, D, 42)
    c.append(L - 1, k, v, starts=ints([0, 400]))
    h = ref.Sequence(Hk, D)
    h.append(f32(k), f32(v))
    K, V = c.read(L - 1, 400, starts=ints([0, 400]), f32=True)
    np.testing.assert_array_equal(f32(K), h.k)
    np.testing.assert_array_equal(f32(V), h.v)
    for new in (1, 40):
        check(nm, c, [h], [new], 16, L - 1, max_new=new)
    q = values(3, 16, D, 43)
    pages = c.select(L - 1, q, 3, starts=ints([0, 3]))
    for i in range(3):
        np.testing.assert_array_equal(pages[i].cpu().numpy(), ref.select(f32(q[i]), h.k[:398 + i], P, 3, 1, 1))
    check(nm, c, [h], [3], 16, L - 1, q=q, pages=pages)


# --- selected pages --------------------------------------------------------------------

def check_select(nm, c, held, new, heads, layer, n, first=1, last=1, seed=5, q=None):
    q = values(sum(new), heads, c.head_dim, seed) if q is None else q
    pages = c.select(layer, q, n, starts=starts_of(new), first=first, last=last)
    assert nm.device_status() == nm.NM_OK
    got, at = pages.cpu().numpy(), 0
    for s, w in enumerate(new):
        for i in range(w):
            m = len(held[s].k) - w + i + 1
            want = ref.select(f32(q[at + i]), held[s].k[:m], c.page_tokens, n, first, last) if m > 0 else np.full(got[0].shape, -1)
            np.testing.assert_array_equal(got[at + i], want, f"sequence {s}, token {i}")
        at += w
    return q, pages


@pytest.mark.parametrize("D,Hk,Hq,P", [(128, 2, 8, 16), (64, 2, 14, 16), (128, 1, 33, 32), (64, 3, 3, 16), (128, 2, 128, 16)])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([17], [1]), ([500], [1]), ([33, 1, 700, 64, 0, 16], [1, 1, 1, 1, 0, 1]),
                                      ([300, 35, 160], [3, 5, 9])])
@pytest.mark.parametrize("n,first,last", [(1, 0, 1), (3, 1, 1), (7, 2, 3), (4, 1, 3)])
def test_select_and_attention_over_it(nm, D, Hk, Hq, P, lens, new, n, first, last):
    c, held = make(nm, lens, P=P, Hk=Hk, D=D, seed=sum(lens))
    q, pages = check_select(nm, c, held, new, Hq, 1, n, first, last)
    check(nm, c, held, new, Hq, 1, q=q, pages=pages)


@pytest.mark.parametrize("D,Hk,Hq,P", [(128, 2, 8, 16), (64, 4, 4, 32)])
def test_select_prompts(nm, D, Hk, Hq, P):
    """Tiles of tokens: many tokens of some sequences, one of others, lists from full to empty."""
    lens, new = [700, 40, 0, 1000, 333], [333, 40, 0, 1, 200]
    c, held = make(nm, lens, P=P, Hk=Hk, D=D, seed=4)
    for n, first, last in ((2, 0, 1), (6, 1, 2), (30, 3, 4)):
        q, pages = check_select(nm, c, held, new, Hq, 1, n, first, last)
        one = torch.cat([c.select(1, q[a:a + 100], n, seqs=ints([0]), starts=ints([0, 100]), first=first, last=last)
                         for a in (233,)])  # few tokens at a time give the same lists
        assert torch.equal(one, pages[233:333])
    check(nm, c, held, new, Hq, 1, q=q, pages=pages)


def test_select_long_and_shared_by_a_cluster(nm):
    """Thousands of pages: one query over several CTAs, ties and all."""
    D, P = 64, 16
    c, held = make(nm, [40000, 20000], P=P, L=1, Hk=1, D=D, seed=6)
    q, pages = check_select(nm, c, held, [1, 1], 4, 0, 100, 2, 3)
    check(nm, c, held, [1, 1], 4, 0, q=q, pages=pages)
    check_select(nm, c, held, [2, 0], 4, 0, 1999, 0, 1, seed=9)


def test_select_ties_go_to_the_lowest_pages(nm):
    """Equal keys in all pages, and a query of zeros: the first of the others are taken."""
    D, P = 128, 16
    k = values(1, 1, D, 1).expand(800, 1, D).contiguous()
    c = nm.Kv8Cache(60, P, 1, 1, D, 1, 60)
    c.reserve(starts=ints([0, 800]))
    c.append(0, k, k, starts=ints([0, 800]))
    for q in (values(1, 4, D, 2), torch.zeros(1, 4, D, dtype=torch.bfloat16, device="cuda")):
        assert c.select(0, q, 9, first=2, last=3).tolist() == [[[0, 1, 2, 3, 4, 5, 47, 48, 49]]]
    assert c.select(0, values(1, 4, D, 2), 50).tolist() == [[list(range(50))]]
    assert c.select(0, values(1, 4, D, 2), 52).tolist() == [[list(range(50)) + [-1, -1]]]


def test_select_edge_queries(nm):
    """Infinities, NaN, huge and tiny values in q; NaN keys in a page."""
    D, P, Hq = 128, 16, 4
    lens = [400]
    c, held = make(nm, lens, P=P, L=1, Hk=1, D=D, seed=21)
    q = values(6, Hq, D, 22)
    q[0, 1, 5], q[1, 0, 0], q[1, 2, 7] = float("nan"), float("inf"), float("-inf")
    q[2] *= 1e30
    q[3] *= 1e-38
    q[4, 0, 0] = 3e38
    q[5] = 1e-42
    check_select(nm, c, held, [6], Hq, 0, 7, 1, 1, q=q)
    k, v = drifting(200, 1, D, 23, P), values(200, 1, D, 24)
    k[37, 0, 3] = float("nan")
    k[48:64] = float("nan")
    c = nm.Kv8Cache(20, P, 1, 1, D, 1, 20)
    c.reserve(starts=ints([0, 200]))
    c.append(0, k, v, starts=ints([0, 200]))
    h = ref.Sequence(1, D)
    h.append(f32(k), f32(v))
    check_select(nm, c, [h], [1], Hq, 0, 5)


def test_attention_over_lists_of_ones_own(nm):
    """Any ascending lists: empty, pages beyond the query, a single old page, all pages."""
    D, P, Hk, Hq = 128, 32, 2, 12
    lens, new = [300, 90], [4, 3]
    c, held = make(nm, lens, P=P, Hk=Hk, D=D, seed=31)
    lists = np.full((7, Hk, 10), -1, np.int32)
    lists[0, 1, :2] = [0, 9]
    lists[1, 0, :1] = [4]
    lists[1, 1, :10] = range(10)
    lists[2, :, :3] = [1, 3, 8]
    lists[4, 0, :1] = [2]  # 88 tokens are seen of 90: its last page in part
    lists[5, :, :3] = [0, 1, 2]
    lists[6, 1, :2] = [0, 2]
    pages = torch.from_numpy(lists).cuda()
    check(nm, c, held, new, Hq, 1, pages=pages)
    # 64 query heads to a kv head: two tiles of rows
    c1, held1 = make(nm, lens, P=P, Hk=1, D=D, seed=32)
    check(nm, c1, held1, new, 64, 1, pages=pages[:, 1:].contiguous())


def test_lists_that_name_nothing_are_reported(nm):
    """Entries out of range or out of order: passed over, and the status tells."""
    D, P = 64, 16
    c, held = make(nm, [100], P=P, Hk=1, D=D, seed=33)
    q = values(1, 4, D, 34)
    good = c.attention(1, q, pages=ints([1, 4, -1]).view(1, 1, 3))
    assert nm.device_status() == nm.NM_OK
    for bad in ([1, 4, 4], [1, 4, 3], [1, 4, 7], [1, 4, 1 << 30], [1, 4, -2]):
        out = c.attention(1, q, pages=ints(bad).view(1, 1, 3))
        assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(out, good), bad
    assert torch.equal(c.attention(1, q, pages=ints([1, 4]).view(1, 1, 2)), good) and nm.device_status() == nm.NM_OK


def test_long_lists_cut_over_many_ctas(nm):
    """One query over hundreds of pages, and many queries at once; results repeat."""
    D, P, Hk, Hq = 128, 16, 2, 8
    c, held = make(nm, [9000, 8000], P=P, L=1, Hk=Hk, D=D, seed=35)
    for new in ([1, 1], [40, 3], [200, 100]):
        q, n = values(sum(new), Hq, D, 36), 150
        pages = c.select(0, q, n, starts=starts_of(new))
        if sum(new) < 100:
            out, lse = check(nm, c, held, new, Hq, 0, q=q, pages=pages)
        else:  # a few of many tokens, each as a sequence's last one would be
            out, lse = c.attention(0, q, starts=starts_of(new), pages=pages, lse=True)
            for t in (0, 99, 199, 200, 299):
                s, m = (0, 8801 + t) if t < 200 else (1, 7901 + t - 200)
                o, l, A, B = ref.attention(f64(q[t:t + 1]), held[s].k[:m].astype(np.float64), held[s].v[:m].astype(np.float64), m,
                                           D ** -0.5, pages[t:t + 1].cpu().numpy(), P)
                e = 2.0 ** -16 * B + 2.0 ** -15
                assert np.all(np.abs(f64(lse[t:t + 1]) - l) <= e)
                tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + m * 2.0 ** -27
                assert np.all(np.abs(f64(out[t:t + 1]) - o) <= tol)
        o2, l2 = c.attention(0, q, starts=starts_of(new), pages=pages, lse=True)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert nm.device_status() == nm.NM_OK


# --- tables, rows of no sequence, pages ------------------------------------------------

def test_rows_of_no_sequence(nm):
    """Padding past the last sequence, and starts out of range: zeros, -inf, -1; other rows as ever."""
    D, Hk, Hq = 128, 2, 8
    c, held = make(nm, [40, 400], P=16, Hk=Hk, D=D, seed=41)
    q = values(7, Hq, D, 42)
    good, gl = c.attention(1, q[:5], starts=ints([0, 2, 5]), lse=True)
    gp = c.select(1, q[:5], 4, starts=ints([0, 2, 5]))
    for out in (torch.full_like(q, 3.0),):
        o, l = c.attention(1, q, starts=ints([0, 2, 5]), out=out, lse=True)
        assert torch.equal(o[:5], good) and bool((o[5:] == 0).all()) and bool(torch.isneginf(l[5:]).all())
    p = c.select(1, q, 4, starts=ints([0, 2, 5]), out=torch.full((7, Hk, 4), 9, dtype=torch.int32, device="cuda"))
    assert torch.equal(p[:5], gp) and bool((p[5:] == -1).all())
    o, l = c.attention(1, q, starts=ints([0, 2, 5]), pages=p, lse=True)
    assert bool((o[5:] == 0).all()) and bool(torch.isneginf(l[5:]).all())
    k, v = c.read(1, 7, starts=ints([0, 2, 5]))
    assert bool((k[5:] == 0).all()) and bool((v[5:] == 0).all())
    many = values(200, 64, D, 43)  # and in the kernel for prompts
    o, l = c.attention(1, many, starts=ints([0, 20, 190]), lse=True, out=torch.full_like(many, 3.0))
    assert bool((o[190:] == 0).all()) and bool(torch.isneginf(l[190:]).all()) and bool(torch.isfinite(l[20:190]).all())
    assert nm.device_status() == nm.NM_OK
    p = c.select(1, q, 4, starts=ints([0, 2, 9]), out=torch.full((7, Hk, 4), 9, dtype=torch.int32, device="cuda"))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(p[:2], gp[:2]) and bool((p[2:] == -1).all())
    o = c.attention(1, q, starts=ints([0, 2, 9]), pages=p)
    assert nm.device_status() == nm.NM_ERR_BOUNDS and bool((o[2:] == 0).all())


def test_tables_out_of_range_are_reported(nm):
    """Ids, lengths and pages out of range: nothing is followed, the status tells, other sequences are right."""
    D, Hk = 128, 2
    c, held = make(nm, [300, 300], P=16, seed=81)
    q = values(2, 8, D, 82)
    good, pages = c.attention(1, q), c.select(1, q, 5)
    assert nm.device_status() == nm.NM_OK
    bad = c.attention(1, q, seqs=ints([0, 2]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(bad[0], good[0]) and bool((bad[1] == 0).all())
    p = c.select(1, q, 5, seqs=ints([0, -1]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(p[0], pages[0]) and bool((p[1] == -1).all())
    saved, pool = c.book.clone(), c.pool.clone()
    c.lens[1] = 1 << 29
    bad = c.attention(1, q, pages=pages)
    assert nm.device_status() == nm.NM_ERR_BOUNDS and bool((bad[1] == 0).all())
    c.book.copy_(saved)
    c.tables[1, 2], c.tables[1, 18] = c.n_pages, -7
    for p in (None, pages):
        bad = c.attention(1, q, pages=p)
        assert bool(torch.isfinite(bad).all())
        if p is None:
            assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(bad[0], good[0])
    many = values(300, 64, D, 83)
    out = c.attention(1, many, seqs=ints([1]), starts=ints([0, 300]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and bool(torch.isfinite(out).all())
    c.select(1, q, 5)
    assert nm.device_status() == nm.NM_ERR_BOUNDS
    k = values(2, Hk, D, 83)
    c.append(1, k, k, seqs=ints([1, 5]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(c.pool, pool)
    kk, _ = c.read(1, 2, seqs=ints([1, 0]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and bool((kk[0] == 0).all())
    c.book.copy_(saved)
    qo = c.append(1, k, k, q=q, rope=rope_table(299, D))  # a rope table that ends before the position
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(c.pool, pool) and bool((qo == 0).all())
    assert torch.equal(c.attention(1, q), good) and nm.device_status() == nm.NM_OK


@pytest.mark.parametrize("max_new,heads", [(1, 8), (64, 64)])
def test_missing_pages_are_not_attended(nm, max_new, heads):
    """A page that the table does not name: its tokens take no part, in each kernel."""
    D, P = 128, 16
    c, held = make(nm, [150], P=P, L=1, Hk=1, D=D, seed=84)
    c.tables[0, 3] = -1
    q = values(40, heads, D, 85)
    out, lse = c.attention(0, q, starts=ints([0, 40]), max_new=max_new, lse=True)
    assert nm.device_status() == nm.NM_ERR_BOUNDS
    lists = np.tile(np.array([0, 1, 2, 4, 5, 6, 7, 8, 9], np.int32), (40, 1, 1))
    o, l, A, B = ref.attention(f64(q), held[0].k.astype(np.float64), held[0].v.astype(np.float64), 150, D ** -0.5, lists, P)
    e = 2.0 ** -16 * B + 2.0 ** -15
    assert np.all(np.abs(f64(lse) - l) <= e)
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + 150 * 2.0 ** -27
    assert np.all(np.abs(f64(out) - o) <= tol)


@pytest.mark.parametrize("seed", range(2))
def test_pages_random_walk(nm, seed):
    """Reserve, fork, free and compact in random order: tables equal the model's, and pool bytes follow."""
    r = np.random.RandomState(seed)
    P = [16, 64][seed]
    n_pages, S, MP, L, Hk, D = [61, 25][seed], 9, 12, 2, 2, 64
    c = nm.Kv8Cache(n_pages, P, L, Hk, D, S, MP)
    c.pool.copy_(torch.from_numpy(r.randint(0, 256, c.pool.shape).astype(np.uint8)))
    m = ref4.Pages(n_pages, P, S, MP)
    pool = c.pool.cpu().numpy().copy()
    cell = 32 * D + 16
    for _ in range(40):
        what = r.randint(4)
        ids = r.permutation(S)[:r.randint(1, 5)].tolist()
        if what == 0:
            new = [int(r.randint(0, 3 * P)) for _ in ids]
            c.reserve(ints(ids), starts_of(new))
            m.reserve(ids, new)
        elif what == 1:
            src = [int(r.randint(S)) for _ in ids]
            dst = [i for i in range(S) if m.lens[i] == 0][:len(src)]
            src = src[:len(dst)]
            c.fork(ints(src), ints(dst))
            m.fork(src, dst)
            v = pool.reshape(n_pages, L * Hk, -1)
            for a, b, tokens in (m.copies if m.result == 0 else []):
                v[b, :, :-(-tokens // 16) * cell] = v[a, :, :-(-tokens // 16) * cell]
        elif what == 2:
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


def test_copy_pages_and_formats(nm):
    a, b = nm.Kv8Cache(7, 32, 3, 2, 64, 1, 4), nm.Kv8Cache(5, 32, 3, 2, 64, 1, 4)
    r = np.random.RandomState(1)
    pa, pb = (r.randint(0, 256, x.pool.shape).astype(np.uint8) for x in (a, b))
    a.pool.copy_(torch.from_numpy(pa))
    b.pool.copy_(torch.from_numpy(pb))
    a.copy_pages(ints([6, 0, 3]), ints([1, 4, 0]), b)
    pb[[1, 4, 0]] = pa[[6, 0, 3]]
    assert np.array_equal(b.pool.cpu().numpy(), pb)
    four = nm.Kv4Cache(5, 32, 3, 2, 64, 1, 4)
    for x, y in ((a, four), (four, a)):
        with pytest.raises(ValueError):
            x.copy_pages(ints([0]), ints([0]), y)


def test_shared_page_is_not_written(nm):
    """After a refused reserve the tokens would fall on a page that a fork shares: nothing is written."""
    D, Hk, P = 128, 2, 16
    c, held = make(nm, [32], P=P, L=1, Hk=Hk, D=D, extra=0, seed=91, max_seqs=2)
    c.fork(ints([0]), ints([1]))
    c.reserve(ints([1]))
    assert c.info.tolist()[1] == 1  # a page is lacking
    pool = c.pool.clone()
    k = values(1, Hk, D, 92)
    c.append(0, k, k, seqs=ints([1]))
    assert nm.device_status() == nm.NM_ERR_BOUNDS and torch.equal(c.pool, pool)


def test_select_arguments(nm):
    c, held = make(nm, [50], P=16, Hk=1, D=64, seed=93)
    q = values(1, 4, 64, 94)
    for kw in (dict(n=4, first=-1), dict(n=4, last=0), dict(n=2, first=2, last=1)):
        with pytest.raises(nm.NmError):
            c.select(1, q, **kw)
    with pytest.raises(nm.NmError):
        c.select(2, q, 4)
    with pytest.raises(ValueError):
        c.select(1, q, 4, out=torch.empty(1, 1, 3, dtype=torch.int32, device="cuda"))
    for p in (ints([0]).view(1, 1, 1).long(), ints([0]), torch.empty(1, 1, 0, dtype=torch.int32, device="cuda")):
        with pytest.raises((TypeError, ValueError)):
            c.attention(1, q, pages=p)


# --- used together -----------------------------------------------------------------------

def test_graph_replays_follow_the_tables(nm):
    """A decode step captured once: reserve, append, select and attention over the selected pages, replayed as the
    sequences grow past several pages."""
    D, Hk, H, P, n = 128, 2, 8, 16, 3
    c, held = make(nm, [30, 60], P=P, L=1, Hk=Hk, extra=10, seed=51)
    k, v, q = (values(2, h, D, 52 + i) for i, h in enumerate((Hk, Hk, H)))
    out, pages = torch.empty_like(q), torch.empty(2, Hk, n, dtype=torch.int32, device="cuda")
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        c.reserve(n=2)
        c.append(0, k, v)
        c.select(0, q, n, out=pages)
        c.attention(0, q, out=out, pages=pages)
    for step in range(4):
        for i, t in enumerate((k, v, q)):
            t.copy_(values(2, t.shape[1], D, 60 + 3 * step + i))
        g.replay()
        for i in range(2):
            held[i].append(f32(k[i:i + 1]), f32(v[i:i + 1]))
            want = ref.select(f32(q[i]), held[i].k, P, n, 1, 1)
            np.testing.assert_array_equal(pages[i].cpu().numpy(), want)
            o, _, A, B = ref.attention(f64(q[i:i + 1]), held[i].k.astype(np.float64), held[i].v.astype(np.float64), len(held[i].k),
                                       D ** -0.5, want[None], P)
            tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2.0 ** -13 + 2.0 ** -15 * B[..., None]) * A + 1e-6
            assert np.all(np.abs(f64(out[i:i + 1]) - o) <= tol)
    assert c.lens.tolist() == [34, 64] and nm.device_status() == nm.NM_OK


def test_fork_decode_compact(nm):
    """Forks share full pages with their bounds; each goes on by itself, with the scale of its own last block; after the
    parent is freed and the pool compacted, selection and attention still find them."""
    D, Hk, P, H = 128, 2, 16, 8
    c, held = make(nm, [86], P=P, L=2, Hk=Hk, extra=12, seed=71, max_seqs=3)
    c.fork(ints([0, 0]), ints([1, 2]))
    held = [held[0], held[0].copy(), held[0].copy()]
    for step in range(12):
        k, v = values(3, Hk, D, 100 + step, 2.0 ** (step % 5)), values(3, Hk, D, 200 + step, 3.0 ** (step % 3))
        k[1] *= 4.0
        c.reserve(ints([0, 1, 2]))
        c.append(1, k, v, seqs=ints([0, 1, 2]))
        for i in range(3):
            held[i].append(f32(k[i:i + 1]), f32(v[i:i + 1]))
    c.free(ints([0]))
    c.compact()
    kk, vv = c.read(1, 196, seqs=ints([1, 2]), starts=ints([0, 98, 196]), f32=True)
    np.testing.assert_array_equal(f32(kk), np.concatenate([held[1].k, held[2].k]))
    np.testing.assert_array_equal(f32(vv), np.concatenate([held[1].v, held[2].v]))
    q = values(2, H, D, 74)
    pages = c.select(1, q, 4, seqs=ints([1, 2]))
    out = c.attention(1, q, seqs=ints([1, 2]), pages=pages)
    for i in (0, 1):
        h = held[i + 1]
        np.testing.assert_array_equal(pages[i].cpu().numpy(), ref.select(f32(q[i]), h.k, P, 4, 1, 1))
        o, _, A, B = ref.attention(f64(q[i:i + 1]), h.k.astype(np.float64), h.v.astype(np.float64), 98, D ** -0.5, pages[i:i + 1].cpu().numpy(), P)
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2.0 ** -13 + 2.0 ** -15 * B[..., None]) * A + 1e-6
        assert np.all(np.abs(f64(out[i:i + 1]) - o) <= tol)
    assert nm.device_status() == nm.NM_OK


@pytest.mark.parametrize("D,Hq", [(128, 4), (64, 8), (128, 13), (64, 16)])
def test_many_lists_a_warp_each(nm, D, Hq):
    """So many tokens that each list is one warp's: sequences that end and begin, padding, empty lists."""
    P = 16
    lens, new = [3000, 900, 40], [900, 400, 40]
    c, held = make(nm, lens, P=P, L=1, Hk=1, D=D, seed=37)
    q = values(1400, Hq, D, 38)
    starts = starts_of(new)  # 60 rows belong to no sequence
    pages = c.select(0, q, 9, starts=starts)
    pages[5] = -1
    pages[950, 0, 3:] = -1
    out, lse = c.attention(0, q, starts=starts, pages=pages, lse=True, out=torch.full_like(q, 7.0))
    assert nm.device_status() == nm.NM_OK
    assert bool((out[1340:] == 0).all()) and bool(torch.isneginf(lse[1340:]).all())
    assert bool((out[5] == 0).all()) and bool(torch.isneginf(lse[5]).all())
    for t in (0, 1, 31, 899, 900, 950, 1299, 1300, 1301, 1339):
        s, m = (0, 2101 + t) if t < 900 else (1, 501 + t - 900) if t < 1300 else (2, 1 + t - 1300)
        o, l, A, B = ref.attention(f64(q[t:t + 1]), held[s].k[:m].astype(np.float64), held[s].v[:m].astype(np.float64), m,
                                   D ** -0.5, pages[t:t + 1].cpu().numpy(), P)
        e = 2.0 ** -16 * B + 2.0 ** -15
        assert np.all(np.abs(f64(lse[t:t + 1]) - l) <= e)
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + m * 2.0 ** -27
        assert np.all(np.abs(f64(out[t:t + 1]) - o) <= tol)
    # each list by itself gives the same to rounding, and calls repeat
    few = torch.cat([c.attention(0, q[t:t + 1], seqs=ints([0]), starts=ints([0, 1]), pages=pages[t:t + 1]) for t in (899,)])
    assert float((few[0].float() - out[899].float()).abs().max()) < 0.05
    o2, l2 = c.attention(0, q, starts=starts, pages=pages, lse=True)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    # entries out of order or range are passed over and reported
    bad = pages.clone()
    bad[7, 0, 4], bad[8, 0, 8] = 1 << 20, 0
    c.attention(0, q, starts=starts, pages=bad)
    assert nm.device_status() == nm.NM_ERR_BOUNDS


@pytest.mark.parametrize("max_new,heads", [(1, 8), (64, 8), (64, 64), (0, 8)])
def test_attention_nonfinite_queries_stay_in_their_rows(nm, max_new, heads):
    """NaN and infinities in q: NaN in that row and no other, in each kernel (0: over lists), and nothing in a row that
    sees no token."""
    c, held = make(nm, [100], seed=92)
    q = values(40, heads, 128, 93)
    kw = dict(pages=c.select(1, q, 3, starts=ints([0, 40]))) if max_new == 0 else dict(max_new=max_new)
    good, gl = c.attention(1, q, starts=ints([0, 40]), lse=True, **kw)
    bad = q.clone()
    bad[7, 3, 11], bad[20, 6, 5], bad[21, 0, 0] = float("nan"), float("inf"), float("-inf")
    out, lse = c.attention(1, bad, starts=ints([0, 40]), lse=True, **kw)
    same = torch.ones(40, heads, dtype=torch.bool, device="cuda")
    for t, h in ((7, 3), (20, 6), (21, 0)):
        same[t, h] = False
        assert bool(torch.isnan(out[t, h]).all()) and bool(torch.isnan(lse[t, h]))
    assert torch.equal(out[same], good[same]) and torch.equal(lse[same], gl[same])
    short = nm.Kv8Cache(3, 16, 1, 2, 128, 1, 3)
    short.reserve(starts=ints([0, 30]))
    k = values(30, 2, 128, 94)
    short.append(0, k, k, starts=ints([0, 30]))
    kw = dict(pages=torch.zeros(40, 2, 1, dtype=torch.int32, device="cuda")) if max_new == 0 else dict(max_new=max_new)
    out, lse = short.attention(0, bad, starts=ints([0, 40]), lse=True, **kw)  # the first ten rows see nothing
    assert bool((out[:10] == 0).all()) and bool(torch.isneginf(lse[:10]).all())
    assert bool(torch.isnan(out[20, 6]).all()) and bool(torch.isfinite(out[19]).all())


@pytest.mark.parametrize("max_new,heads", [(1, 8), (64, 64), (0, 8)])
def test_attention_queries_of_wide_range(nm, max_new, heads):
    """Channels of q from the row's largest down to 2^-24 of it, in an order that meets large keys: q is exact
    above 2^-13 of the largest and off by at most 2^-21 of it below, so scores are off by at most 2^-21 max |q| sum |k| more."""
    c, held = make(nm, [300], Hk=2, seed=95)
    g = torch.Generator().manual_seed(96)
    q = (torch.randn(30, heads, 128, generator=g) * torch.exp2(-24 * torch.rand(30, heads, 128, generator=g)) * 30).bfloat16().cuda()
    kw = dict(pages=c.select(1, q, 5, starts=ints([0, 30]))) if max_new == 0 else dict(max_new=max_new)
    out, lse = c.attention(1, q, starts=ints([0, 30]), lse=True, **kw)
    K, V = held[0].k.astype(np.float64), held[0].v.astype(np.float64)
    lists = kw["pages"].cpu().numpy() if max_new == 0 else None
    o, l, A, B = ref.attention(f64(q), K, V, 300, 128 ** -0.5, lists, 32)
    e = 2.0 ** -16 * B + 2.0 ** -15 + 2.0 ** -21 * np.abs(f64(q)).max(-1) * np.abs(K).sum(-1).max() * 128 ** -0.5
    assert np.all(np.abs(f64(lse) - l) <= e)
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + 300 * 2.0 ** -27
    assert np.all(np.abs(f64(out) - o) <= tol)
    assert nm.device_status() == nm.NM_OK


@pytest.mark.parametrize("n", [0, 2, 100])
def test_example_decode_loop(nm, n):
    """The example's loop over the 8-bit cache, all of it (0), two selected pages, and more pages than there are:
    every attention result against the definition, on the q, k, v that went in."""
    from examples import paged_decode as ex
    P = 16
    d = ex.Decoder(layers=2, hidden=256, heads=8, kv_heads=2, dim=64, ffn=512, sequences=3, tokens=80, page=P, seed=5, bits=8, pages=n)
    g = torch.Generator(device="cuda").manual_seed(6)
    prompt = torch.randn(53, 256, generator=g, device="cuda").bfloat16()
    traces, step = [], d.step

    def traced(x, seqs, starts=None):
        t = []
        y = step(x, seqs, starts, trace=t)
        traces.append((seqs.tolist(), None if starts is None else starts.tolist(), t))
        return y

    d.step = traced
    out = ex.run(d, prompt, 3, 14)
    assert len(out) == 14 and nm.device_status() == nm.NM_OK
    rope = d.rope.cpu().numpy()
    held = [[ref.Sequence(2, 64) for _ in range(2)] for _ in range(3)]  # [sequence][layer]
    for seqs, starts, layers in traces:
        if starts is None and len(held[1][0].k) == 0:  # the fork came before the first joint step
            for s in (1, 2):
                held[s] = [h.copy() for h in held[0]]
        starts = starts or list(range(len(seqs) + 1))
        for layer, (q, k, v, a) in enumerate(layers):
            q, k, v = (f32(t).reshape(t.shape[0], -1, 64) for t in (q, k, v))
            for i, s in enumerate(seqs):
                h = held[s][layer]
                rows = slice(starts[i], starts[i + 1])
                pos = np.arange(len(h.k), len(h.k) + starts[i + 1] - starts[i])
                cos, sin = rope[pos, :32], rope[pos, 32:]
                h.append(ref.rotate(k[rows], cos, sin), v[rows])
                rq = ref.bf16(ref.rotate(q[rows], cos, sin))
                m = len(h.k) - len(rq)
                lists = np.array([ref.select(rq[j], h.k[:m + j + 1], P, n, 1, 1) for j in range(len(rq))]) if n else None
                o, _, A, B = ref.attention(rq.astype(np.float64), h.k.astype(np.float64), h.v.astype(np.float64), len(h.k), 0.125, lists, P)
                e = 2.0 ** -16 * B[..., None] + 2.0 ** -15
                tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e + 2.0 ** -14) * A + 1e-6
                assert np.all(np.abs(f64(a[rows]).reshape(o.shape) - o) <= tol)
    assert d.cache.lens.tolist() == [67, 0, 0] and d.cache.info.tolist()[:2] == [d.cache.n_pages - 5, 0]


def test_two_caches_on_two_streams(nm):
    """Calls with caches of their own may overlap: each on a stream, alternating, as often as it takes to meet."""
    D, P, H = 128, 64, 8
    both = [make(nm, [3000, 700], P=P, Hk=2, D=D, seed=61 + i) for i in range(2)]
    q = [values(2, H, D, 63 + i) for i in range(2)]
    many = [values(300, H, D, 65 + i) for i in range(2)]
    st = starts_of([250, 50])
    want = [(c.attention(1, q[i]), c.select(1, q[i], 9), c.attention(1, many[i], starts=st)) for i, (c, _) in enumerate(both)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, (c, _) in enumerate(both):
            with torch.cuda.stream(streams[i]):
                got[i].append((c.attention(1, q[i]), c.select(1, q[i], 9), c.attention(1, many[i], starts=st)))
    torch.cuda.synchronize()
    for i in range(2):
        for x in got[i]:
            for a, b in zip(x, want[i]):
                assert torch.equal(a, b)
    assert nm.device_status() == nm.NM_OK


@pytest.mark.parametrize("D", [64, 128])
def test_page_filled_and_selected_in_one_call(nm, D):
    """Drafted tokens that fill a page and go on: later ones of the call select it by its new bounds; appended again
    (after a rejection the tokens are written anew) the bounds follow."""
    P, Hk, H = 16, 1, 4
    c, held = make(nm, [205, 260], P=P, L=1, Hk=Hk, D=D, extra=4, seed=97)  # the second: for a table of more pages
    one = ints([0])
    rope = rope_table(230, D)
    cs = rope.cpu().numpy()
    c.reserve(one, ints([0, 20]))
    for seed in (1, 2):
        h = held[0].copy()
        k, v, q = values(20, Hk, D, 100 * seed, 2.0 * seed), values(20, Hk, D, 100 * seed + 1), values(20, H, D, 100 * seed + 2)
        q = c.append(0, k, v, q=q, rope=rope, seqs=one, starts=ints([0, 20]))
        cos, sin = cs[205:225, :D // 2], cs[205:225, D // 2:]
        if seed == 2:  # a scale does not shrink until its block's first position is written again
            h.e[12] = e_before
            h.k[192:205], h.v[192:205] = kept
        h.append(ref.rotate(f32(k), cos, sin), f32(v))
        e_before, kept = h.e[12].copy(), (h.k[192:205].copy(), h.v[192:205].copy())
        kk, vv = c.read(0, 225, one, ints([0, 225]), f32=True)
        np.testing.assert_array_equal(f32(kk), h.k)
        np.testing.assert_array_equal(f32(vv), h.v)
        for n in (3, 6):
            pages = c.select(0, q, n, one, ints([0, 20]))
            for t in range(20):
                np.testing.assert_array_equal(pages[t].cpu().numpy(), ref.select(f32(q[t]), h.k[:206 + t], P, n, 1, 1))
    assert nm.device_status() == nm.NM_OK


@pytest.mark.parametrize("D,P,Hq", [(128, 64, 8), (64, 32, 10), (128, 32, 3)])
def test_many_lists_of_pages_of_several_cells(nm, D, P, Hq):
    """A warp's cells come two at a time: lists of odd and even length, pages that end inside a pair, a page that the
    table does not name, and NaN in whatever lies behind the last token."""
    c, held = make(nm, [1200, 2 * P + 17], P=P, L=1, Hk=1, D=D, extra=1, seed=41)
    new = [1000, 2 * P + 17]
    T = sum(new)
    q = values(T, Hq, D, 42)
    starts = starts_of(new)
    pages = c.select(0, q, 5, starts=starts)
    pages[10:200, 0, 3:] = -1
    pages[200:300, 0, 1:] = -1
    q[40, 1, 3] = float("inf")
    out, lse = c.attention(0, q, starts=starts, pages=pages, lse=True)
    assert nm.device_status() == nm.NM_OK
    assert bool(torch.isnan(out[40, 1]).all()) and int(torch.isnan(out).sum()) == D
    q[40, 1, 3] = 0.0

    def right(t, s, m, listed, out, lse):
        o, l, A, B = ref.attention(f64(q[t:t + 1]), held[s].k[:m].astype(np.float64), held[s].v[:m].astype(np.float64), m,
                                   D ** -0.5, listed, P)
        e = 2.0 ** -16 * B + 2.0 ** -15
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + m * 2.0 ** -27
        return np.all(np.abs(f64(lse[t:t + 1]) - l) <= e) and np.all(np.abs(f64(out[t:t + 1]) - o) <= tol)

    for t in [0, 9, 10, 41, 199, 200, 299, 300, 999] + list(range(1000, T)):
        s, m = (0, 201 + t) if t < 1000 else (1, t - 999)
        assert right(t, s, m, pages[t:t + 1].cpu().numpy(), out, lse), t
    c.tables[0, 0] = -1  # as if page 0 were not listed
    o2, l2 = c.attention(0, q, starts=starts, pages=pages, lse=True)
    assert nm.device_status() == nm.NM_ERR_BOUNDS
    assert torch.equal(o2[1000:], out[1000:])
    for t in (0, 10, 300, 999):
        rest = pages[t:t + 1].cpu().numpy()
        rest = np.concatenate([rest[..., 1:], np.full_like(rest[..., :1], -1)], -1) if rest[0, 0, 0] == 0 else rest
        assert right(t, 0, 201 + t, rest, o2, l2), t


def test_a_thousand_sequences_and_one_listed_often(nm):
    """1024 sequences in one call of each kind and kernel, and a sequence that a call lists more than once: each
    listing is answered as by itself."""
    D, P, Hk, H, S = 64, 16, 1, 8, 1024
    r = np.random.RandomState(7)
    lens = [int(x) for x in r.randint(0, 40, S)]
    c, held = make(nm, lens, P=P, L=1, Hk=Hk, D=D, extra=S, seed=101, max_seqs=S)  # a page more for each
    k, v, q = values(S, Hk, D, 102), values(S, Hk, D, 103), values(S, H, D, 104)
    c.reserve(n=S)
    assert c.info[1] == 0
    c.append(0, k, v)
    for i, h in enumerate(held):
        h.append(f32(k[i:i + 1]), f32(v[i:i + 1]))
    lists = c.select(0, q, 2)
    out, part = c.attention(0, q), c.attention(0, q, pages=lists)
    kk, vv = c.read(0, S, f32=True)
    long = [i for i in range(S) if lens[i] >= 3]
    starts = starts_of([3 if n >= 3 else 0 for n in lens])  # drafted tokens of most of them
    q3 = values(int(starts[-1]), H, D, 105)
    few = c.attention(0, q3, starts=starts, max_new=3)
    lists3 = c.select(0, q3, 2, starts=starts)
    part3 = c.attention(0, q3, starts=starts, pages=lists3)
    q9 = q3.repeat(1, 6, 1)  # 48 heads and no bound on the new tokens: the kernel for prompts
    many = c.attention(0, q9, starts=starts)
    assert nm.device_status() == nm.NM_OK

    def right(got, q, i, m, listed=None):
        o, _, A, B = ref.attention(f64(q), held[i].k[:m].astype(np.float64), held[i].v[:m].astype(np.float64), m, D ** -0.5,
                                   listed, P)
        e = 2.0 ** -16 * B + 2.0 ** -15
        return np.all(np.abs(f64(got) - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + m * 2.0 ** -27)

    for i in r.choice(S, 60, replace=False).tolist() + [0, S - 1]:
        n = lens[i] + 1
        np.testing.assert_array_equal(f32(kk[i]), held[i].k[-1])
        np.testing.assert_array_equal(f32(vv[i]), held[i].v[-1])
        np.testing.assert_array_equal(lists[i].cpu().numpy(), ref.select(f32(q[i]), held[i].k, P, 2, 1, 1))
        assert right(out[i:i + 1], q[i:i + 1], i, n) and right(part[i:i + 1], q[i:i + 1], i, n, lists[i:i + 1].cpu().numpy())
        for t in range(int(starts[i]), int(starts[i + 1])):
            m = n - 2 + t - int(starts[i])
            np.testing.assert_array_equal(lists3[t].cpu().numpy(), ref.select(f32(q3[t]), held[i].k[:m], P, 2, 1, 1))
            assert right(few[t:t + 1], q3[t:t + 1], i, m) and right(many[t:t + 1], q9[t:t + 1], i, m)
            assert right(part3[t:t + 1], q3[t:t + 1], i, m, lists3[t:t + 1].cpu().numpy())
    ids = [long[0], long[1], long[0], long[0], long[2]]  # one sequence three times
    again = c.attention(0, q[:5], seqs=ints(ids))
    la = c.select(0, q[:5], 2, seqs=ints(ids))
    pa = c.attention(0, q[:5], seqs=ints(ids), pages=la)
    ka, _ = c.read(0, 5, seqs=ints(ids), f32=True)
    for j, i in enumerate(ids):
        n = lens[i] + 1
        assert right(again[j:j + 1], q[j:j + 1], i, n) and right(pa[j:j + 1], q[j:j + 1], i, n, la[j:j + 1].cpu().numpy())
        np.testing.assert_array_equal(f32(ka[j]), held[i].k[-1])
    q5 = values(15, 48, D, 106)
    m5 = c.attention(0, q5, seqs=ints(ids), starts=ints([0, 3, 6, 9, 12, 15]))
    for j, i in enumerate(ids):
        assert right(m5[3 * j + 2:3 * j + 3], q5[3 * j + 2:3 * j + 3], i, lens[i] + 1)
    assert nm.device_status() == nm.NM_OK


def test_prompt_and_lists_captured_and_replayed(nm):
    """The kernels for prompts and for many lists in one graph, replayed while the lengths and the rows' cuts change."""
    D, P, Hk, H = 128, 16, 2, 32
    c, held = make(nm, [700, 300], P=P, L=1, Hk=Hk, D=D, seed=111)
    q = values(900, H, D, 112)
    starts, pages = starts_of([700, 200]), torch.empty(900, Hk, 7, dtype=torch.int32, device="cuda")
    out, part = torch.empty_like(q), torch.empty_like(q)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        c.attention(0, q, starts=starts, out=out)
        c.select(0, q, 7, starts=starts, out=pages)
        c.attention(0, q, starts=starts, pages=pages, out=part)
    for new, drop in (([700, 200], 0), ([1, 300], 0), ([600, 300], 100), ([0, 0], 0), ([650, 250], 0)):
        c.lens[0] = 700 - drop
        starts.copy_(starts_of(new))
        out.fill_(3.0), part.fill_(3.0), pages.fill_(9)
        g.replay()
        assert nm.device_status() == nm.NM_OK
        n = sum(new)
        assert bool((out[n:] == 0).all()) and bool((part[n:] == 0).all()) and bool((pages[n:] == -1).all())
        at = 0
        for i, m in enumerate(new):
            L = len(held[i].k) - (drop if i == 0 else 0)
            for t in sorted({0, 1, m // 2, m - 1} & set(range(m))):
                pos, x = L - m + t, at + t
                for got, listed in ((out, None), (part, pages[x:x + 1].cpu().numpy())):
                    o, _, A, B = ref.attention(f64(q[x:x + 1]), held[i].k[:pos + 1].astype(np.float64),
                                               held[i].v[:pos + 1].astype(np.float64), pos + 1, D ** -0.5, listed, P)
                    e = 2.0 ** -16 * B + 2.0 ** -15
                    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2 * e[..., None] + 2.0 ** -14) * A + (pos + 1) * 2.0 ** -27
                    assert np.all(np.abs(f64(got[x:x + 1]) - o) <= tol)
                np.testing.assert_array_equal(listed[0], ref.select(f32(q[x]), held[i].k[:pos + 1], P, 7, 1, 1))
            at += m


def test_prompts_and_many_lists_past_4_gib(nm):
    """The kernels for prompts, for tiles of tokens and for many lists over pages whose bytes lie past 2^32 of the pool."""
    P, L, Hk, D = 128, 32, 8, 128
    per = nm.lib().nm_kv8_page_bytes(P, L, Hk, D)
    n = (1 << 32) // per + 8
    c = nm.Kv8Cache(n, P, L, Hk, D, 1, 4)
    c.refs.fill_(1)  # only the last four pages are free
    c.refs[n - 4:] = 0
    c.info[0] = 4
    c.reserve(starts=ints([0, 500]))
    k, v = values(500, Hk, D, 141), values(500, Hk, D, 142)
    c.append(L - 1, k, v, starts=ints([0, 500]))
    h = ref.Sequence(Hk, D)
    h.append(f32(k), f32(v))
    check(nm, c, [h], [120], 16, L - 1, max_new=120)  # 240 rows, 1920 in all
    q, pages = check_select(nm, c, [h], [120], 16, L - 1, 3)
    check(nm, c, [h], [120], 16, L - 1, q=q, pages=pages)
    assert int(c.tables[0, 0]) == n - 4 and (n - 4) * per > 1 << 32
