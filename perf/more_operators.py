"""Cases of the 8-bit paged KV cache: append, attention, and attention over selected pages.

Each case is run in a plain form (elementary torch operations in fp32) or, with
``own`` set, through the package's Kv8Cache. Both work on the same buffers:

* ``pool``: uint8 [pages][page bytes]; a page holds, per layer and kv head, ``page / 16`` cells of 16
  tokens and then the page's bounds. A cell is [K codes][V codes][scale of K, scale of V (fp32), 8 bytes]:
  codes are 8-bit floats (4 exponent, 3 mantissa bits), scales powers of two for all 16 tokens. Bounds
  are int8 [D] upper, int8 [D] lower, an fp32 step and 12 bytes; a page has them once it is full.
* ``book``: int32 [info 16][lens][refs][tables], each part padded to 4 ints.
"""
import functools

import torch

own = False

DEV = "cuda"
CELL = 16
LIMIT = 32768.0
CODE = torch.float8_e4m3fn


# --- cases ----------------------------------------------------------------------

def _attn(name, heads, kv, dim, page, lens, new=None, layers=1):
    return {"name": name, "op": "attention", "heads": heads, "kv_heads": kv, "dim": dim, "page": page, "layers": layers,
            "lens": ",".join(map(str, lens)), "new": ",".join(map(str, new or [1] * len(lens)))}


def _append(name, heads, kv, dim, page, lens, new=None, layers=1):
    return {**_attn(name, heads, kv, dim, page, lens, new, layers), "op": "append"}


def _sparse(name, heads, kv, dim, page, lens, new, pages, first=1, last=2):
    return {**_attn(name, heads, kv, dim, page, lens, new), "op": "sparse", "pages": pages, "first": first, "last": last}


def listed():
    return [
        # a decode step early in a chat: one short sequence, 8B head layout; latency counts
        _attn("decode_1x129", 32, 8, 128, 64, [129]),
        # a decode step of the largest batch the linears take, contexts of all lengths
        _attn("decode_8_ragged", 32, 8, 128, 64, [8191, 1, 4097, 613, 2048, 7777, 100, 3333], layers=2),
        # a decode step at the end of a long document, 70B head layout
        _attn("decode_1x131071", 64, 8, 128, 64, [131071]),
        # checking five drafted tokens a sequence in one pass, 14B head layout (five query heads to a kv head)
        _attn("verify_4x5", 40, 8, 128, 32, [16385, 9001, 12288, 15000], [5, 5, 5, 5]),
        # one pass over mixed prompts: a 512-token chunk behind a long context, and two new prompts
        _attn("prompts_ragged", 32, 8, 128, 64, [16896, 2777, 333], [512, 2777, 333]),
        # a whole prompt at once
        _attn("prompt_8192", 32, 8, 128, 64, [8192], [8192]),
        # the cache write of a decode step at batch 8, and the blocks it touched read back
        _append("append_step_8", 32, 8, 128, 64, [8192, 2, 4098, 614, 2049, 7778, 101, 3334], layers=2),
        # the cache write of a long prompt, and the values read back
        _append("append_prompt_16384", 32, 8, 128, 64, [16384], [16384]),
        # a decode step that reads 2048 of 131071 tokens, 70B head layout
        _sparse("sparse_1x131071", 64, 8, 128, 64, [131071], [1], 32),
        # a batch whose long sequences are read in part and whose short ones in full
        _sparse("sparse_8_ragged", 32, 8, 128, 64, [40000, 1, 9001, 613, 32768, 17777, 100, 65535], [1] * 8, 24),
        # drafted tokens, each with pages of its own, 14B head layout
        _sparse("sparse_verify_4x5", 40, 8, 128, 32, [16385, 9001, 12288, 15000], [5, 5, 5, 5], 40),
        # a 512-token chunk of a prompt behind 16384 tokens, each token with pages of its own
        _sparse("sparse_chunk_512", 32, 8, 128, 64, [16896], [512], 16),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["decode", "decode", "verify", "prompt", "prompt", "append", "append", "sparse", "sparse"])
    heads, kv = rng.choice([(32, 8), (40, 8), (64, 8), (8, 8), (14, 2), (16, 1)])
    dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if kind == "decode":
        n = rng.randint(1, 8)
        return _unnamed(_attn("", heads, kv, dim, page, [_log(rng, 1, 100000 // n) for _ in range(n)], layers=rng.randint(1, 2)))
    if kind == "verify":
        n = rng.randint(1, 6)
        new = [rng.randint(1, 12) for _ in range(n)]
        return _unnamed(_attn("", heads, kv, dim, page, [w + _log(rng, 1, 60000 // n) for w in new], new))
    if kind == "sparse":
        n = rng.randint(1, 6)
        new = [_log(rng, 1, 200 // n)] * n if rng.random() < 0.4 else [1] * n
        lens = [w + _log(rng, 1, 60000 // n) for w in new]
        pages = _log(rng, 3, 64)
        first = rng.randint(0, 2)
        return _unnamed(_sparse("", heads, kv, dim, page, lens, new, pages, first, rng.randint(1, max(1, min(4, pages - first)))))
    n = rng.randint(1, 4)
    heads, kv = rng.choice([(32, 8), (40, 8), (8, 8), (14, 2), (16, 1)])
    new = [_log(rng, 1 if kind == "append" else 17, 6000 // n) for _ in range(n)]
    lens = [w + rng.choice([0, 0, _log(rng, 1, 6000 // n)]) for w in new]
    return _unnamed((_append if kind == "append" else _attn)("", heads, kv, dim, page, lens, new, rng.randint(1, 2)))


def _unnamed(c):
    return {k: v for k, v in c.items() if k != "name"}


def _ints(text):
    return [int(t) for t in text.split(",")]


def _cell_bytes(dim):
    return 2 * CELL * dim + 16


def _head_bytes(dim, page):
    return page // CELL * _cell_bytes(dim) + 2 * dim + 16


def _read_back(lens, new):
    # the new tokens, and those before them that can share their first block
    return [min(n, w + CELL - 1) for n, w in zip(lens, new)]


def work(case):
    H, Hk, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens, new = _ints(case["lens"]), _ints(case["new"])
    T, per = sum(new), 2 * D + 0.5  # codes and scales of a token and kv head
    if case["op"] == "append":
        # q read and written, k and v read, the rotation table, the codes and bounds written, the values read back
        back = sum(_read_back(lens, new))
        return {"bytes": int(T * (4 * H * D + 4 * Hk * D + 4 * D + Hk * (per + (2 * D + 4) / P)) + back * Hk * (per + 4 * D)),
                "flops": T * (H + Hk) * D * 4 + T * Hk * D * 4}
    if case["op"] == "attention":
        seen = sum(w * (n - w) + w * (w + 1) // 2 for n, w in zip(lens, new))
        return {"bytes": int(sum(lens) * Hk * per) + T * H * (4 * D + 4), "flops": 4 * D * H * seen}
    read = bounds = seen = scored = 0
    for n, w in zip(lens, new):
        pages = [(n - w + i) // P + 1 for i in range(w)]
        most = [min(x, case["pages"]) * P for x in pages]
        read += min(n, sum(most))
        bounds += n // P if pages[-1] > case["pages"] else 0
        seen += sum(min(m, n - w + i + 1) for i, m in enumerate(most))
        scored += sum(x for x in pages if x > case["pages"])
    return {"bytes": int(read * Hk * per) + bounds * Hk * (2 * D + 4) + T * (H * (4 * D + 4) + 4 * Hk * case["pages"]),
            "flops": 4 * D * H * seen + 4 * D * Hk * scored}


# --- the layout ------------------------------------------------------------------

@functools.lru_cache(None)
def _offsets(dim):
    """Byte offsets in a cell of the codes of K and of V, each [16 tokens][dim]."""
    tok = torch.arange(CELL, device=DEV)[:, None]
    ch = torch.arange(dim, device=DEV)[None, :]
    k = (tok // 8) * (8 * dim) + (ch // 64) * 512 + (tok % 8) * 64 + ch % 64
    v = CELL * dim + (ch // 32) * 512 + (ch % 32) // 4 * 64 + (tok % 8) // 2 * 16 + (ch % 4) * 4 + tok % 2 + 2 * (tok // 8)
    return k, v


def _exponent(most, significand, exponent):
    """The least e with most <= significand * 2^(exponent + e), significand in [0.5, 1)."""
    f, k = torch.frexp(most)
    return k - exponent + (f > significand).int()


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _cells_of(pool, dims, page, layer, cell):
    """Cells [n][H][cell bytes] (a copy) and their byte offsets in the pool [n][H]."""
    L, H, D, P = dims
    base = (page * (L * H) + layer * H)[:, None] + torch.arange(H, device=DEV)
    base = base * _head_bytes(D, P) + (cell * _cell_bytes(D))[:, None]
    return pool.view(-1)[base[..., None] + torch.arange(_cell_bytes(D), device=DEV)], base


def _write(pool, tables, layer, dims, seq, pos, k, v):
    """Appends the tokens (sequence seq[i], position pos[i], fp32 k, v [T][H][D]): their blocks' scales grow where
    they have to, the codes held there are re-expressed, and the bounds of the pages that fill up are written."""
    L, H, D, P = dims
    ok = torch.isfinite(k).all(-1) & torch.isfinite(v).all(-1)  # [T][H]
    k, v = (torch.where(ok[..., None], x.clamp(-LIMIT, LIMIT), torch.zeros_like(x)) for x in (k, v))
    width = tables.shape[1] * (P // CELL)
    block, at = torch.unique(seq * width + pos // CELL, return_inverse=True)
    n = block.numel()
    first = torch.full((n,), CELL, dtype=torch.long, device=DEV).scatter_reduce(0, at, pos % CELL, "amin")
    page = tables[block // width, block % width // (P // CELL)].long()
    cells, base = _cells_of(pool, dims, page, layer, block % (P // CELL))
    scales = cells[..., 2 * CELL * D:2 * CELL * D + 8].contiguous().view(torch.float32)  # [n][H][2]
    for i, (x, off) in enumerate(zip((k, v), _offsets(D))):
        most = torch.zeros(n, H, device=DEV).scatter_reduce(0, at[:, None].expand(-1, H), x.abs().amax(-1), "amax")
        e = torch.where(most > 0, _exponent(most, 0.875, 9), torch.full_like(most, -24, dtype=torch.int32)).clamp(-24, 7)
        held = (first > 0)[:, None]
        old = torch.where(held, scales[..., i], torch.zeros_like(most))
        s = torch.maximum(_pow2(e), old)
        codes = cells[:, :, off.flatten()].view(n, H, CELL, D)
        again = (codes.view(CODE).float() * (old / s)[..., None, None]).to(CODE).view(torch.uint8)
        grown = (held & (s > old))[..., None, None]
        codes = torch.where(grown, again, codes)
        new = (x / s[at][..., None]).to(CODE).view(torch.uint8)
        if i == 0:
            new = torch.where(ok[..., None], new, torch.full_like(new, 0x7F))
        codes[at, :, pos % CELL] = new
        cells[:, :, off.flatten()] = codes.view(n, H, -1)
        scales[..., i] = s
    cells[..., 2 * CELL * D:2 * CELL * D + 8] = scales.view(torch.uint8)
    pool.view(-1)[base[..., None] + torch.arange(_cell_bytes(D), device=DEV)] = cells
    full = pos % P == P - 1
    if bool(full.any()):
        _write_bounds(pool, layer, dims, tables[seq[full], pos[full] // P].long())


def _bounds_of(pool, layer, dims, pages):
    """Bounds of full pages, from the keys they hold: upper, lower (whole numbers in fp32 [n][H][D]), step [n][H]."""
    K = _gather(pool, pages[:, None], layer, dims)[0]  # [n][H][P][D]
    nan = torch.isnan(K)
    hi = torch.where(nan, torch.full_like(K, -1e30), K).amax(2)
    lo = torch.where(nan, torch.full_like(K, 1e30), K).amin(2)
    hi, lo = torch.where(hi < lo, torch.zeros_like(hi), hi), torch.where(hi < lo, torch.zeros_like(lo), lo)
    most = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    e = torch.where(most > 0, _exponent(most, 127 / 128, 7), torch.full_like(most, -30, dtype=torch.int32)).clamp(min=-30)
    step = _pow2(e)
    return torch.ceil(hi / step[..., None]), torch.floor(lo / step[..., None]), step


def _write_bounds(pool, layer, dims, pages):
    L, H, D, P = dims
    for part in pages.split(256):
        hi, lo, step = _bounds_of(pool, layer, dims, part)
        tail = torch.cat([hi.to(torch.int8).view(torch.uint8), lo.to(torch.int8).view(torch.uint8),
                          step[..., None].contiguous().view(torch.uint8)], -1)
        base = ((part * (L * H) + layer * H)[:, None] + torch.arange(H, device=DEV) + 1) * _head_bytes(D, P) - 2 * D - 16
        pool.view(-1)[base[..., None] + torch.arange(2 * D + 4, device=DEV)] = tail


def _gather(pool, pages, layer, dims):
    """fp32 K, V [n][H][m * P][D] held by pages [n][m]."""
    L, H, D, P = dims
    heads = pool.view(-1, L, H, _head_bytes(D, P))[pages, layer]  # [n][m][H][head bytes]
    cells = heads[..., :P // CELL * _cell_bytes(D)].unflatten(-1, (P // CELL, _cell_bytes(D))).permute(0, 2, 1, 3, 4)
    n, _, m = cells.shape[:3]
    scales = cells[..., 2 * CELL * D:2 * CELL * D + 8].contiguous().view(torch.float32)
    out = []
    for i, off in enumerate(_offsets(D)):
        x = cells[..., off.flatten()].view(CODE).float() * scales[..., i:i + 1]
        out.append(x.reshape(n, H, m * P, D))
    return out


# --- states ------------------------------------------------------------------------

def _pad4(n):
    return -(-n // 4) * 4


def _kv_values(T, H, D, g):
    """Keys with a few large, offset channels per head (as rotary models have) and plain values, in bf16."""
    k = torch.randn(T, H, D, generator=g, device=DEV)
    scale = 0.5 + torch.rand(H, D, generator=g, device=DEV)
    scale[:, ::37] *= 4.0
    shift = torch.randn(H, D, generator=g, device=DEV) * 0.5
    # tokens near one another are alike, so that pages differ
    drift = torch.randn(-(-T // 48), H, D, generator=g, device=DEV).repeat_interleave(48, 0)[:T]
    return ((k + drift) * scale + shift).bfloat16(), torch.randn(T, H, D, generator=g, device=DEV).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    H, Hk, D, P, L = case["heads"], case["kv_heads"], case["dim"], case["page"], case["layers"]
    lens, new = _ints(case["lens"]), _ints(case["new"])
    n, T = len(lens), sum(new)
    need = [-(-x // P) for x in lens]
    n_pages, max_pages = sum(need) + 3, max(need) + 1
    per = L * Hk * _head_bytes(D, P)
    st = {"case": case, "layer": L - 1, "lens_host": lens, "new_host": new, "max_pages": max_pages}
    st["pool"] = torch.randint(0, 256, (n_pages, per), generator=g, device=DEV, dtype=torch.uint8)
    a, b, c = 16, _pad4(n), _pad4(n_pages)
    st["book"] = torch.zeros(a + b + c + _pad4(n * max_pages), dtype=torch.int32, device=DEV)
    info, lens_t, refs = st["book"][:a], st["book"][a:a + n], st["book"][a + b:a + b + n_pages]
    tables = _tables_of(st)[1]
    tables.fill_(-1)
    perm = torch.randperm(n_pages, generator=g, device=DEV).int()
    at = 0
    for s in range(n):
        tables[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
        lens_t[s] = lens[s]
    refs[perm[:at].long()] = 1
    info[0] = n_pages - at

    def starts(counts):
        return torch.tensor([sum(counts[:i]) for i in range(n + 1)], dtype=torch.int32, device=DEV)

    st["starts"] = None if max(new) == 1 and min(new) == 1 else starts(new)
    st["q"] = torch.randn(T, H, D, generator=g, device=DEV).bfloat16()
    if case["op"] == "append":
        st["k"], st["v"] = _kv_values(T, Hk, D, g)
        inv = 500000.0 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
        ang = torch.arange(max(lens), device=DEV, dtype=torch.float64)[:, None] * inv
        st["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        st["back"], st["back_starts"] = sum(_read_back(lens, new)), starts(_read_back(lens, new))
    for s in range(n):
        end = lens[s] - (new[s] if case["op"] == "append" else 0)
        for x in range(0, end, 32768):
            y = min(end, x + 32768)
            pos = torch.arange(x, y, device=DEV)
            k, v = _kv_values(y - x, Hk, D, g)
            _write(st["pool"], tables, L - 1, (L, Hk, D, P), torch.full_like(pos, s), pos, k.float(), v.float())
    return st


def _tables_of(st):
    n, pages = len(st["lens_host"]), st["pool"].shape[0]
    at = 16 + _pad4(n) + _pad4(pages)
    return st["book"][16:16 + n], st["book"][at:at + n * st["max_pages"]].view(n, st["max_pages"])


def _tokens_of(st):
    """(sequence, position) of each new token."""
    lens, _ = _tables_of(st)
    n, new = len(st["lens_host"]), st["new_host"]
    if st["starts"] is None:
        return torch.arange(n, device=DEV), (lens - 1).long()
    starts = st["starts"].long()
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), starts[1:] - starts[:-1], output_size=sum(new))
    return seq, lens[seq].long() - starts[1:][seq] + torch.arange(sum(new), device=DEV)


# --- one pass ------------------------------------------------------------------------

def _cache(st):
    """The handle a user's program keeps over its buffers."""
    if "cache" not in st:
        import sparse_decoding_gb300 as nm
        c = st["case"]
        st["cache"] = nm.Kv8Cache(st["pool"].shape[0], c["page"], c["layers"], c["kv_heads"], c["dim"],
                                  max_seqs=len(st["lens_host"]), max_pages=st["max_pages"], pool=st["pool"], book=st["book"])
    return st["cache"]


def run(st):
    return (_OWN if own else _PLAIN)[st["case"]["op"]](st)


def _own_attention(st):
    out, lse = _cache(st).attention(st["layer"], st["q"], starts=st["starts"], max_new=max(st["new_host"]), lse=True)
    return {"out": out, "lse": lse}


def _own_append(st):
    c = _cache(st)
    q = c.append(st["layer"], st["k"], st["v"], q=st["q"], rope=st["rope"], starts=st["starts"])
    k, v = c.read(st["layer"], st["back"], starts=st["back_starts"])
    return {"q": q, "k": k, "v": v}


def _own_sparse(st):
    c, case = _cache(st), st["case"]
    pages = c.select(st["layer"], st["q"], case["pages"], starts=st["starts"], first=case["first"], last=case["last"])
    out, lse = c.attention(st["layer"], st["q"], starts=st["starts"], pages=pages, lse=True)
    return {"pages": pages, "out": out, "lse": lse}


def _weigh(S, see, V, scale):
    """softmax(scale S) V over the columns that `see` allows, and the log of the sums; 0 and -inf where there are none."""
    S *= scale
    S.masked_fill_(~see, float("-inf"))
    m = S.amax(-1, keepdim=True).clamp(min=-1e30)
    S -= m
    S.exp_()
    z = S.sum(-1, keepdim=True)
    out = (S @ V) / torch.where(z > 0, z, torch.ones_like(z))
    return out, torch.where(z > 0, m + torch.log(z), torch.full_like(z, float("-inf")))[..., 0]


def _plain_attention(st):
    c = st["case"]
    H, Hk, D, P, L = c["heads"], c["kv_heads"], c["dim"], c["page"], c["layers"]
    lens, tables = _tables_of(st)
    n, r = len(st["lens_host"]), H // Hk
    most, width = max(st["lens_host"]), max(st["new_host"])
    pages = tables[:, :-(-most // P)].clamp(min=0).long()
    K, V = _gather(st["pool"], pages, st["layer"], (L, Hk, D, P))
    K, V = K[:, :, :most], V[:, :, :most]
    at = torch.arange(most, device=DEV)
    V = torch.where((at[None] < lens[:, None])[:, None, :, None], V, torch.zeros_like(V))
    seq, pos = _tokens_of(st)
    first = st["starts"].long()[:-1] if st["starts"] is not None else torch.arange(n, device=DEV)
    i = torch.arange(seq.numel(), device=DEV) - first[seq]
    q = torch.zeros(n, width, H, D, device=DEV)
    q[seq, i] = st["q"].float()
    q = q.view(n, width, Hk, r, D).permute(0, 2, 1, 3, 4).reshape(n, Hk, width * r, D)
    last = torch.full((n, width), -1, dtype=torch.long, device=DEV)
    last[seq, i] = pos
    see = at[None, None] <= last.repeat_interleave(r, 1)[:, :, None]  # [n][width * r][most]
    out, lse = _weigh(q @ K.transpose(-1, -2), see[:, None], V, D ** -0.5)
    out = out.view(n, Hk, width, r, D).permute(0, 2, 1, 3, 4).reshape(n, width, H, D)
    lse = lse.view(n, Hk, width, r).permute(0, 2, 1, 3).reshape(n, width, H)
    return {"out": out[seq, i].bfloat16(), "lse": lse[seq, i].contiguous()}


def _rotate(x, cos, sin):
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(st):
    c = st["case"]
    dims = (c["layers"], c["kv_heads"], c["dim"], c["page"])
    Hk, D, P = dims[1:]
    lens, tables = _tables_of(st)
    seq, pos = _tokens_of(st)
    cos, sin = st["rope"][pos][:, None].chunk(2, -1)
    q = _rotate(st["q"].float(), cos, sin).bfloat16()
    _write(st["pool"], tables, st["layer"], dims, seq, pos, _rotate(st["k"].float(), cos, sin), st["v"].float())
    # read back the blocks that hold the tokens
    starts = st["back_starts"].long()
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), starts[1:] - starts[:-1], output_size=st["back"])
    pos = lens[seq].long() - starts[1:][seq] + torch.arange(st["back"], device=DEV)
    cells, _ = _cells_of(st["pool"], dims, tables[seq, pos // P].long(), st["layer"], pos % P // CELL)
    scales = cells[..., 2 * CELL * D:2 * CELL * D + 8].contiguous().view(torch.float32)
    kv = []
    for i, off in enumerate(_offsets(D)):
        codes = torch.gather(cells, 2, off[pos % CELL][:, None].expand(-1, Hk, -1))
        kv.append((codes.view(CODE).float() * scales[..., i:i + 1]).bfloat16())
    return {"q": q, "k": kv[0], "v": kv[1]}


def _plain_select(st, seq, pos):
    """The pages of each new token and kv head, int32 [T][Hk][pages]: ascending, -1 behind."""
    c = st["case"]
    H, Hk, D, P, L = c["heads"], c["kv_heads"], c["dim"], c["page"], c["layers"]
    want, first, last = c["pages"], c["first"], c["last"]
    _, tables = _tables_of(st)
    q = st["q"].float()
    q = torch.where(torch.isfinite(q), q, torch.zeros_like(q)).view(-1, Hk, H // Hk, D)
    up, down = torch.zeros_like(q[:, :, 0]), torch.zeros_like(q[:, :, 0])
    for h in range(H // Hk):
        up, down = up + q[:, :, h].clamp(min=0), down + q[:, :, h].clamp(max=0)
    most = torch.maximum(up, -down).amax(-1)
    e = torch.where(most > 0, _exponent(most, 127 / 128, 7), torch.zeros_like(most, dtype=torch.int32))
    up, down = (torch.round(torch.ldexp(x, -e[..., None])) for x in (up, down))
    count = (pos // P + 1)[:, None, None]
    width = -(-max(st["lens_host"]) // P)
    score = torch.full((len(seq), Hk, max(width, want)), float("-inf"), device=DEV)
    for s in range(len(st["lens_host"])):
        rows = torch.nonzero(seq == s).flatten()
        m = st["lens_host"][s] // P  # full pages
        for x in range(0, m, 4096):
            y = min(m, x + 4096)
            hi, lo, step = _bounds_of(st["pool"], st["layer"], (L, Hk, D, P), tables[s, x:y].long())
            part = up[rows].transpose(0, 1) @ hi.permute(1, 2, 0) + down[rows].transpose(0, 1) @ lo.permute(1, 2, 0)  # [Hk][rows][m]
            score[rows, :, x:y] = (part * step.T[:, None]).transpose(0, 1)
    at = torch.arange(score.shape[-1], device=DEV)
    score = torch.where((at < first) | (at >= count - last), torch.full_like(score, float("inf")), score)
    score = torch.where(at < count, score, torch.full_like(score, float("-inf")))
    best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :want]
    best = torch.where(best < count, best, torch.full_like(best, 1 << 30)).sort(-1).values
    return torch.where(best < 1 << 30, best, torch.full_like(best, -1)).int()


def _plain_sparse(st):
    c = st["case"]
    H, Hk, D, P, L = c["heads"], c["kv_heads"], c["dim"], c["page"], c["layers"]
    _, tables = _tables_of(st)
    seq, pos = _tokens_of(st)
    pages = _plain_select(st, seq, pos)
    heads = st["pool"].view(-1, L, Hk, _head_bytes(D, P))
    out = torch.empty(len(seq), H, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(len(seq), H, device=DEV)
    step = max(1, (1 << 28) // (Hk * c["pages"] * P * D))
    hk = torch.arange(Hk, device=DEV)[:, None]
    for a in range(0, len(seq), step):
        z = slice(a, a + step)
        mine = pages[z].long()
        phys = tables[seq[z, None, None], mine.clamp(min=0)].long()
        raw = heads[phys, st["layer"], hk][..., :P // CELL * _cell_bytes(D)].unflatten(-1, (P // CELL, _cell_bytes(D)))
        scales = raw[..., 2 * CELL * D:2 * CELL * D + 8].contiguous().view(torch.float32)
        K, V = ((raw[..., off.flatten()].view(CODE).float() * scales[..., i:i + 1]).reshape(len(mine), Hk, -1, D)
                for i, off in enumerate(_offsets(D)))
        t = mine[..., None] * P + torch.arange(P, device=DEV)
        see = ((mine[..., None] >= 0) & (t <= pos[z, None, None, None])).flatten(2)
        V = torch.where(see[..., None], V, torch.zeros_like(V))
        q = st["q"][z].float().view(-1, Hk, H // Hk, D)
        o, l = _weigh(q @ K.transpose(-1, -2), see[:, :, None], V, D ** -0.5)
        out[z], lse[z] = o.reshape(-1, H, D).bfloat16(), l.reshape(-1, H)
    return {"pages": pages, "out": out, "lse": lse}


_OWN = {"attention": _own_attention, "append": _own_append, "sparse": _own_sparse}
_PLAIN = {"attention": _plain_attention, "append": _plain_append, "sparse": _plain_sparse}


# --- the definition in 64 bits ----------------------------------------------------------

def _stored(st, s, h, n):
    """K, V (fp64 [n][D]) of one kv head of a sequence, straight from the format's definition."""
    c, pool = st["case"], st["pool"]
    D, P, L, H = c["dim"], c["page"], c["layers"], c["kv_heads"]
    size, cell = P // 16 * (32 * D + 16) + 2 * D + 16, 32 * D + 16
    t = torch.arange(n, device=DEV)
    page = _tables_of(st)[1][s, t // P].long()
    base = ((page * L + st["layer"]) * H + h) * size + t % P // 16 * cell
    flat, w, ch = pool.view(-1), (t % 16)[:, None], torch.arange(D, device=DEV)[None]
    # K: two halves of eight tokens, in pieces of 64 channels; V: 16-byte pieces of 4 channels x (tokens 2j, 2j+1, 2j+8, 2j+9)
    kb = w // 8 * 8 * D + ch // 64 * 512 + w % 8 * 64 + ch % 64
    vb = 16 * D + ch // 4 * 64 + w % 8 // 2 * 16 + ch % 4 * 4 + w // 8 * 2 + w % 2
    scale = pool.view(torch.float32).view(-1)
    out = []
    for i, at in enumerate((kb, vb)):
        b = flat[base[:, None] + at].to(torch.int64)
        e, m = b // 8 % 16, (b % 8).double()
        x = torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)
        x = torch.where(b % 128 == 127, torch.full_like(x, float("nan")), x)
        out.append(torch.where(b > 127, -x, x) * scale[(base + 32 * D) // 4 + i].double()[:, None])
    return out


def _exact_append(st):
    c = st["case"]
    Hk, D = c["kv_heads"], c["dim"]
    lens, new, half = st["lens_host"], st["new_host"], D // 2
    back = _read_back(lens, new)
    pos = torch.cat([torch.arange(a - b, a, device=DEV) for a, b in zip(lens, new)])
    angle = st["rope"][pos].double()[:, None]

    def turned(x):
        x = x.double()
        y = torch.empty_like(x)
        y[..., :half] = x[..., :half] * angle[..., :half] - x[..., half:] * angle[..., half:]
        y[..., half:] = x[..., half:] * angle[..., :half] + x[..., :half] * angle[..., half:]
        return y

    def rounded(x, s):  # to three mantissa bits above 2^-6 of the scale, to 2^-9 of it below
        x = x / s
        step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(x / step) * step * s

    res, at = {"q": turned(st["q"]), "k": [], "v": []}, 0
    k, v = turned(st["k"]), st["v"].double()
    for s, (n, w) in enumerate(zip(lens, new)):
        held = [[x[:, None] for x in _stored(st, s, h, n - w)] for h in range(Hk)]
        for name, fresh, i in (("k", k, 0), ("v", v, 1)):
            x = torch.cat([torch.cat([p[i] for p in held], 1), fresh[at:at + w]])
            begin = (n - w) // 16 * 16  # the blocks from here on are written
            out = x.clone()
            for b in range(begin, n, 16):
                whole = x[b:b + 16]
                top = whole.abs().amax((0, 2), keepdim=True)
                sc = torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-24, 7))
                out[b:b + 16] = rounded(whole, sc)
                if b < n - w:  # held under a larger scale already: it stays
                    old = _scale_of(st, s, b, i)[None, :, None]
                    out[b:b + 16] = rounded(whole, torch.maximum(sc, old))
            res[name].append(out[n - back[s]:])
        at += w
    return {"q": res["q"], "k": torch.cat(res["k"]), "v": torch.cat(res["v"])}


def _scale_of(st, s, token, i):
    c = st["case"]
    D, P, L, H = c["dim"], c["page"], c["layers"], c["kv_heads"]
    size = P // 16 * (32 * D + 16) + 2 * D + 16
    page = int(_tables_of(st)[1][s, token // P])
    at = ((page * L + st["layer"]) * H + torch.arange(H, device=DEV)) * size + token % P // 16 * (32 * D + 16) + 32 * D
    return st["pool"].view(torch.float32).view(-1)[at // 4 + i].double()


def _exact_pages(case, K, q, n):
    """The pages of the last w queries of a sequence of n tokens, for one kv head: K its keys [n][D], q [w][r][D]."""
    P, want, w = case["page"], case["pages"], q.shape[0]
    m = n // P  # full pages
    pages = K[:m * P].view(m, P, K.shape[-1])
    hi, lo = pages.amax(1), pages.amin(1)
    step = torch.exp2(torch.ceil(torch.log2(torch.maximum(hi.abs(), lo.abs()).amax(-1) / 127)).clamp(min=-30))
    up, down = q.clamp(min=0).sum(1), q.clamp(max=0).sum(1)
    unit = torch.exp2(torch.ceil(torch.log2(torch.maximum(up, -down).amax(-1, keepdim=True) / 127)))
    score = torch.round(up / unit) @ torch.ceil(hi / step[:, None]).T + torch.round(down / unit) @ torch.floor(lo / step[:, None]).T
    score = (score * step).tolist()  # whole numbers below 2^24 times a power of two: exact
    out = []
    for i in range(w):
        count = (n - w + i) // P + 1
        forced = [z for z in range(count) if count <= want or z < case["first"] or z >= count - case["last"]]
        rest = sorted(set(range(count)) - set(forced), key=lambda z: (-score[i][z], z))
        mine = sorted(forced + rest[:want - len(forced)])
        out.append(mine + [-1] * (want - len(mine)))
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def exact(case, seed):
    H, Hk, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens, new = _ints(case["lens"]), _ints(case["new"])
    if case["op"] == "append" and sum(new) > 20000:
        return None
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    out = torch.zeros(sum(new), H, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(sum(new), H, dtype=torch.float64, device=DEV)
    pages = torch.full((sum(new), Hk, case.get("pages", 1)), -1, dtype=torch.int32, device=DEV)
    at, r = 0, H // Hk
    for s, (n, w) in enumerate(zip(lens, new)):
        q = st["q"][at:at + w].double()
        t = torch.arange(n, device=DEV)
        hidden = t[None] > torch.arange(n - w, n, device=DEV)[:, None]
        for h in range(Hk):
            K, V = _stored(st, s, h, n)
            unseen = hidden
            if case["op"] == "sparse":
                mine = _exact_pages(case, K, q[:, h * r:(h + 1) * r], n)
                pages[at:at + w, h] = mine
                keep = torch.zeros(w, -(-n // P) + 1, dtype=torch.bool, device=DEV)  # the last column: no page
                keep.scatter_(1, torch.where(mine < 0, -(-n // P), mine).long(), True)
                unseen = hidden | ~keep[:, t // P]
            for j in range(h * r, (h + 1) * r):
                x = (q[:, j] @ K.T / D ** 0.5).masked_fill(unseen, float("-inf"))
                lse[at:at + w, j] = torch.logsumexp(x, -1)
                out[at:at + w, j] = torch.softmax(x, -1) @ V
        at += w
    res = {"out": out, "lse": lse}
    return {"pages": pages, **res} if case["op"] == "sparse" else res
