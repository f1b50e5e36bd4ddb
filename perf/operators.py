"""Cases of the 4-bit paged KV cache: append, attention, fork/free/reserve, compact.

Each case is run in a plain form (elementary torch operations in fp32) or, with
``own`` set, through the package's Kv4Cache. Both work on the same buffers:

* ``pool``: uint8 [pages][page bytes]; a page holds, per layer and kv head,
  ``page / 16`` cells of 16 tokens. A cell is [K codes][V codes][K params]
  [V params]; one group of 64 channels of one token has 64 4-bit codes and two
  fp16 parameters (scale, mid): value = mid + scale * (code - 8).
* ``book``: int32 [info 16][lens][refs][tables], each part padded to 4 ints.
"""
import functools

import torch

own = False

DEV = "cuda"
CELL = 16
GROUP = 64
LIMIT = 32768.0


# --- cases ----------------------------------------------------------------------

def _attn(name, heads, kv, dim, page, lens, new=None, layers=1):
    return {"name": name, "op": "attention", "heads": heads, "kv_heads": kv, "dim": dim, "page": page, "layers": layers,
         "lens": ",".join(map(str, lens)), "new": ",".join(map(str, new or [1] * len(lens)))}


def _append(name, heads, kv, dim, page, lens, new=None, layers=1):
    return {**_attn(name, heads, kv, dim, page, lens, new, layers), "op": "append"}


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
        # the cache write of a decode step at batch 8, and the values it holds read back
        _append("append_step_8", 32, 8, 128, 64, [8192, 2, 4098, 614, 2049, 7778, 101, 3334], layers=2),
        # the cache write of a long prompt, and the values read back
        _append("append_prompt_16384", 32, 8, 128, 64, [16384], [16384]),
        # a sampling tree of a small model: drop three branches, fork three anew, make room for a token each
        {"name": "fork_3_small", "op": "fork", "kv_heads": 4, "dim": 64, "page": 16, "layers": 4, "len": 201, "width": 3, "pages": 64},
        # a beam step of the 8B model: drop seven beams, fork seven from the best, make room for a token each
        {"name": "fork_7_8b", "op": "fork", "kv_heads": 8, "dim": 128, "page": 64, "layers": 32, "len": 2031, "width": 7, "pages": 96},
        # a small cache with a few holes
        {"name": "compact_small", "op": "compact", "kv_heads": 4, "dim": 64, "page": 32, "layers": 4, "pages": 200, "live": 120, "seqs": 16},
        # a serving cache of the 8B model half emptied by finished sequences
        {"name": "compact_8b", "op": "compact", "kv_heads": 8, "dim": 128, "page": 64, "layers": 32, "pages": 512, "live": 250, "seqs": 24},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["decode", "decode", "verify", "prompt", "prompt", "append", "append", "fork", "compact"])
    heads, kv = rng.choice([(32, 8), (40, 8), (64, 8), (8, 8), (14, 2), (16, 1)])
    dim, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if kind == "decode":
        n = rng.randint(1, 8)
        return _unnamed(_attn("", heads, kv, dim, page, [_log(rng, 1, 100000 // n) for _ in range(n)], layers=rng.randint(1, 2)))
    if kind == "verify":
        n = rng.randint(1, 6)
        new = [rng.randint(1, 12) for _ in range(n)]
        return _unnamed(_attn("", heads, kv, dim, page, [w + _log(rng, 1, 60000 // n) for w in new], new))
    if kind in ("prompt", "append"):
        n = rng.randint(1, 4)
        heads, kv = rng.choice([(32, 8), (40, 8), (8, 8), (14, 2), (16, 1)])
        new = [_log(rng, 1 if kind == "append" else 17, 6000 // n) for _ in range(n)]
        lens = [w + rng.choice([0, 0, _log(rng, 1, 6000 // n)]) for w in new]
        return _unnamed((_append if kind == "append" else _attn)("", heads, kv, dim, page, lens, new, rng.randint(1, 2)))
    if kind == "fork":
        width, length = rng.randint(1, 12), _log(rng, 1, 4000)
        return {"op": "fork", "kv_heads": kv, "dim": dim, "page": page, "layers": rng.randint(1, 16), "len": length,
                "width": width, "pages": -(-length // page) + 2 * width + rng.randint(1, 40)}
    pages = _log(rng, 24, 400)
    return {"op": "compact", "kv_heads": kv, "dim": dim, "page": page, "layers": rng.randint(1, 16), "pages": pages,
            "live": max(1, int(pages * rng.uniform(0.1, 0.9))), "seqs": rng.randint(1, 8)}


def _unnamed(c):
    return {k: v for k, v in c.items() if k != "name"}


def _ints(text):
    return [int(t) for t in text.split(",")]


def _cell_bytes(dim):
    return CELL * dim + CELL * (dim // GROUP) * 8


def work(case):
    cell = _cell_bytes(case["dim"])
    if case["op"] in ("attention", "append"):
        H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
        lens, new = _ints(case["lens"]), _ints(case["new"])
        T = sum(new)
        if case["op"] == "attention":
            seen = sum(w * (n - w) + w * (w + 1) // 2 for n, w in zip(lens, new))
            return {"bytes": sum(lens) * Hk * cell // CELL + T * H * (4 * D + 4), "flops": 4 * D * H * seen}
        # q read and written, k and v read, the rotation table, the cache written, the values read back
        return {"bytes": T * (4 * H * D + 4 * Hk * D + 4 * D + 2 * Hk * cell // CELL + 4 * Hk * D), "flops": T * (H + Hk) * D * 4 + T * Hk * D * 8}
    per_page = case["layers"] * case["kv_heads"] * cell * (case["page"] // CELL)
    if case["op"] == "fork":
        rem = case["len"] % case["page"]
        per = case["layers"] * case["kv_heads"] * cell * -(-rem // CELL)
        book = 4 * (case["pages"] + 2 * (case["width"] + 1) * (-(-(case["len"] + 1) // case["page"]) + 1))
        return {"bytes": (1 + case["width"]) * per + book, "flops": 0}
    return {"bytes": 2 * _moved(case) * per_page + 8 * case["pages"], "flops": 0}


def _moved(case):
    # the live pages are spread evenly (see _live_pages): those past the live count move
    return int((_live_pages(case) >= case["live"]).sum())


def _live_pages(case):
    # a fixed scatter of `live` pages over the pool: the whole numbers i with the smallest (i * 7919 + 13) mod 10007
    i = torch.arange(case["pages"])
    return torch.sort(torch.argsort((i * 7919 + 13) % 10007, stable=True)[:case["live"]]).values


# --- the layout ------------------------------------------------------------------

@functools.lru_cache(None)
def _offsets(dim):
    """Byte offsets in a cell: K codes [16][dim/2], V codes [16][dim/2] (byte b: channels 2b, 2b+1), K params
    [16][groups][scale, mid], V params [8 token pairs][groups][scale, scale, mid, mid]."""
    G = dim // GROUP
    tok = torch.arange(CELL, device=DEV)[:, None]
    b = torch.arange(dim // 2, device=DEV)[None, :]
    grp, in_group = b // 32, (b % 32)
    k = tok * (dim // 2) + (in_group // 8) * (8 * G) + grp * 8 + in_group % 8
    g8, quad, byte = in_group // 4, (in_group // 2) % 2, in_group % 2
    v = (CELL * dim // 2 + grp * 512 + (g8 * 4 + (tok // 2) % 4) * 16 + (tok // 8) * 8 + quad * 4 + (tok % 2) * 2 + byte)
    t4 = torch.arange(CELL, device=DEV).view(CELL, 1, 1, 1)
    g4 = torch.arange(G, device=DEV).view(1, G, 1, 1)
    w4 = torch.arange(2, device=DEV).view(1, 1, 2, 1)
    b4 = torch.arange(2, device=DEV).view(1, 1, 1, 2)
    kp = CELL * dim + (t4 * G + g4) * 4 + w4 * 2 + b4
    vp = CELL * dim + CELL * G * 4 + ((t4 // 2) * G + g4) * 8 + w4 * 4 + (t4 % 2) * 2 + b4
    return k, v, kp, vp


def _quantise(k, v):
    """fp32 k, v [T][H][D] -> codes (uint8) and fp16 params [T][H][G][2] of each."""
    bad = ~(torch.isfinite(k).all(-1) & torch.isfinite(v).all(-1))
    out = []
    for x in (k, v):
        x = torch.nan_to_num(x, nan=0.0, posinf=LIMIT, neginf=-LIMIT).clamp(-LIMIT, LIMIT)
        g = x.view(*x.shape[:-1], -1, GROUP)
        lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
        s = ((hi - lo) / 15.0).bfloat16().half()  # eight significant bits
        s32 = s.float()
        mid = (lo + s32 * 8.0).half()
        u = torch.where(s32 > 0, torch.round((g - mid.float()) / torch.where(s32 > 0, s32, torch.ones_like(s32))), torch.zeros_like(g))
        out += [(u.clamp(-8, 7) + 8).to(torch.uint8).view(x.shape), torch.cat([s, mid], -1)]
    out[0] = torch.where(bad[..., None], torch.full_like(out[0], 8), out[0])
    out[1] = torch.where(bad[..., None, None], torch.full_like(out[1], float("nan")), out[1])
    return out


def _write(pool, tables, layer, dims, seq, pos, k, v):
    """Writes the tokens (sequence seq[i], position pos[i], fp32 k, v [T][H][D]) into the pool."""
    L, H, D, P = dims
    cb = _cell_bytes(D)
    kc, kp, vc, vp = _quantise(k, v)
    page = tables[seq, pos // P].long()
    base = ((page * L + layer) * H)[:, None] + torch.arange(H, device=DEV)
    base = (base * (P // CELL) + ((pos % P) // CELL)[:, None]) * cb
    off = _offsets(D)
    flat, slot = pool.view(-1), pos % CELL
    for codes, o in ((kc, off[0]), (vc, off[1])):
        flat[base[:, :, None] + o[slot][:, None]] = codes[..., 0::2] | (codes[..., 1::2] << 4)
    for par, o in ((kp, off[2]), (vp, off[3])):
        flat[base[:, :, None] + o[slot].flatten(1)[:, None]] = par.contiguous().view(torch.uint8).flatten(2)


def _gather(pool, pages, layer, dims):
    """fp32 K, V [n][H][pages * P][D] of the sequences whose pages are pages [n][np]."""
    L, H, D, P = dims
    cells = pool.view(-1, L, H, P // CELL, _cell_bytes(D))[pages, layer]  # [n][np][H][P/16][cell]
    cells = cells.permute(0, 2, 1, 3, 4)
    n, _, m = cells.shape[:3]
    out = []
    off = _offsets(D)
    for o, p in ((off[0], off[2]), (off[1], off[3])):
        by = cells[..., o]
        u = torch.stack([by & 15, by >> 4], -1).flatten(-2).float()
        par = cells[..., p].contiguous().view(torch.float16).squeeze(-1).float()  # [...][16][G][2]
        x = (u.view(*u.shape[:-1], -1, GROUP) - 8.0) * par[..., 0:1] + par[..., 1:2]
        out.append(x.reshape(n, H, m * P, D))
    return out


# --- states ------------------------------------------------------------------------

def _pad4(n):
    return -(-n // 4) * 4


def _book(n_pages, max_seqs, max_pages):
    """The int32 bookkeeping buffer and its parts (views): info, lens, refs, tables."""
    a, b, c = 16, _pad4(max_seqs), _pad4(n_pages)
    book = torch.zeros(a + b + c + _pad4(max_seqs * max_pages), dtype=torch.int32, device=DEV)
    parts = book[:a], book[a:a + max_seqs], book[a + b:a + b + n_pages], book[a + b + c:][:max_seqs * max_pages].view(max_seqs, max_pages)
    parts[3].fill_(-1)
    parts[0][0] = n_pages
    return (book, *parts)


def _pool(n_pages, L, H, D, P, g):
    per = L * H * (P // CELL) * _cell_bytes(D)
    return torch.randint(0, 256, (n_pages, per), generator=g, device=DEV, dtype=torch.uint8)


def _kv_values(T, H, D, g):
    """Keys with a few large, offset channels per head (as rotary models have) and plain values, in bf16."""
    k = torch.randn(T, H, D, generator=g, device=DEV)
    scale = 0.5 + torch.rand(H, D, generator=g, device=DEV)
    scale[:, ::37] *= 4.0
    shift = torch.randn(H, D, generator=g, device=DEV) * 0.5
    return (k * scale + shift).bfloat16(), torch.randn(T, H, D, generator=g, device=DEV).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] == "fork":
        return _prepare_fork(case, g)
    if case["op"] == "compact":
        return _prepare_compact(case, g)
    H, Hk, D, P, L = case["heads"], case["kv_heads"], case["dim"], case["page"], case["layers"]
    lens, new = _ints(case["lens"]), _ints(case["new"])
    n, T = len(lens), sum(new)
    need = [-(-x // P) for x in lens]
    n_pages, max_pages = sum(need) + 3, max(need) + 1
    st = {"case": case, "layer": L - 1, "lens_host": lens, "new_host": new}
    st["pool"] = _pool(n_pages, L, Hk, D, P, g)
    st["book"], info, lens_t, refs, tables = _book(n_pages, n, max_pages)
    perm = torch.randperm(n_pages, generator=g, device=DEV).int()
    at = 0
    for s in range(n):
        tables[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
        lens_t[s] = lens[s]
    refs[perm[:at].long()] = 1
    info[0] = n_pages - at
    st["starts"] = None if max(new) == 1 and min(new) == 1 else torch.tensor([sum(new[:i]) for i in range(n + 1)], dtype=torch.int32, device=DEV)
    st["q"] = torch.randn(T, H, D, generator=g, device=DEV).bfloat16()
    if case["op"] == "append":
        st["k"], st["v"] = _kv_values(T, Hk, D, g)
        inv = 500000.0 ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
        ang = torch.arange(max(lens), device=DEV, dtype=torch.float64)[:, None] * inv
        st["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        return st
    for s in range(n):
        for a in range(0, lens[s], 32768):
            b = min(lens[s], a + 32768)
            pos = torch.arange(a, b, device=DEV)
            k, v = _kv_values(b - a, Hk, D, g)
            _write(st["pool"], tables, L - 1, (L, Hk, D, P), torch.full_like(pos, s), pos, k.float(), v.float())
    return st


def _prepare_fork(case, g):
    P, L, Hk, D, n, width = case["page"], case["layers"], case["kv_heads"], case["dim"], case["len"], case["width"]
    max_pages = -(-(n + 1) // P) + 1
    st = {"case": case, "pool": _pool(case["pages"], L, Hk, D, P, g)}
    st["book"], info, lens, refs, tables = _book(case["pages"], width + 1, max_pages)
    perm = torch.randperm(case["pages"], generator=g, device=DEV).int()
    need = -(-n // P)
    tables[0, :need] = perm[:need]
    refs[perm[:need].long()] = 1
    lens[0] = n
    info[0] = case["pages"] - need
    st["src"] = torch.zeros(width, dtype=torch.int32, device=DEV)
    st["dst"] = torch.arange(1, width + 1, dtype=torch.int32, device=DEV)
    st["shape"] = (case["pages"], width + 1, max_pages)
    return st


def _prepare_compact(case, g):
    P, L, Hk, D, pages, seqs = case["page"], case["layers"], case["kv_heads"], case["dim"], case["pages"], case["seqs"]
    st = {"case": case, "pool": _pool(pages, L, Hk, D, P, g)}
    live = _live_pages(case).to(DEV)
    order = live[torch.randperm(case["live"], generator=g, device=DEV)].int()
    max_pages = -(-case["live"] // seqs) + 1
    st["book"], info, lens, refs, tables = _book(pages, seqs, max_pages)
    # the sequences take turns; the first page of sequence 0 is shared by all that have room
    for s in range(seqs):
        mine = order[s::seqs]
        tables[s, :len(mine)] = mine
        lens[s] = len(mine) * P
    refs[live] = 1
    if seqs > 1:
        shared = tables[0, 0].long()
        row = tables[1]
        if int(row[0]) >= 0:
            at = int((row >= 0).sum())
            row[at] = shared
            lens[1] += P
            refs[shared] += 1
    info[0] = pages - case["live"]
    st["saved"] = st["book"].clone()
    st["shape"] = (pages, seqs, max_pages)
    return st


def _views(st):
    pages, seqs, max_pages = st["shape"]
    a, b, c = 16, _pad4(seqs), _pad4(pages)
    book = st["book"]
    return book[:a], book[a:a + seqs], book[a + b:a + b + pages], book[a + b + c:][:seqs * max_pages].view(seqs, max_pages)


# --- one pass ------------------------------------------------------------------------

def _cache(st):
    """The handle a user's program keeps over its buffers."""
    if "cache" not in st:
        import sparse_decoding_gb300 as nm
        c = st["case"]
        st["cache"] = nm.Kv4Cache(st["pool"].shape[0], c["page"], c["layers"], c["kv_heads"], c["dim"],
                                  max_seqs=st["shape"][1] if "shape" in st else len(st["lens_host"]),
                                  max_pages=st["shape"][2] if "shape" in st else max(-(-x // c["page"]) for x in st["lens_host"]) + 1,
                                  pool=st["pool"], book=st["book"])
    return st["cache"]


def run(st):
    return (_OWN if own else _PLAIN)[st["case"]["op"]](st)


def _own_attention(st):
    out, lse = _cache(st).attention(st["layer"], st["q"], starts=st["starts"], max_new=max(st["new_host"]), lse=True)
    return {"out": out, "lse": lse}


def _own_append(st):
    c = _cache(st)
    q = c.append(st["layer"], st["k"], st["v"], q=st["q"], rope=st["rope"], starts=st["starts"])
    k, v = c.read(st["layer"], st["k"].shape[0], starts=st["starts"])
    return {"q": q, "k": k, "v": v}


def _own_fork(st):
    c = _cache(st)
    c.free(st["dst"])
    c.fork(st["src"], st["dst"])
    c.reserve(st["dst"])
    return {"pool": st["pool"], "book": st["book"]}


def _own_compact(st):
    st["book"].copy_(st["saved"])  # so that a pass finds the holes again
    _cache(st).compact()
    return {"pool": st["pool"], "book": st["book"]}


def _tables_of(st):
    c = st["case"]
    n, pages = len(st["lens_host"]), st["pool"].shape[0]
    max_pages = max(-(-x // c["page"]) for x in st["lens_host"]) + 1
    at = 16 + _pad4(n)
    return st["book"][16:16 + n], st["book"][at + _pad4(pages):][:n * max_pages].view(n, max_pages)


def _tokens_of(st):
    """(sequence, position) of each new token."""
    lens, _ = _tables_of(st)
    n, new = len(st["lens_host"]), st["new_host"]
    if st["starts"] is None:
        seq = torch.arange(n, device=DEV)
        return seq, (lens - 1).long()
    starts = st["starts"].long()
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), starts[1:] - starts[:-1], output_size=sum(new))
    i = torch.arange(sum(new), device=DEV) - starts[seq]
    return seq, lens[seq].long() - (starts[1:] - starts[:-1])[seq] + i


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
    S = q @ K.transpose(-1, -2)
    S *= D ** -0.5
    see = at[None, None] <= last.repeat_interleave(r, 1)[:, :, None]  # [n][width * r][most]
    S.masked_fill_(~see[:, None], float("-inf"))
    m = S.amax(-1, keepdim=True).clamp(min=-1e30)
    S -= m
    S.exp_()
    z = S.sum(-1, keepdim=True)
    out = (S @ V) / torch.where(z > 0, z, torch.ones_like(z))
    lse = torch.where(z > 0, m + torch.log(z), torch.full_like(z, float("-inf")))
    out = out.view(n, Hk, width, r, D).permute(0, 2, 1, 3, 4).reshape(n, width, H, D)
    lse = lse.view(n, Hk, width, r).permute(0, 2, 1, 3).reshape(n, width, H)
    return {"out": out[seq, i].bfloat16(), "lse": lse[seq, i]}


def _rotate(x, cos, sin):
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(st):
    c = st["case"]
    Hk, D, P, L = c["kv_heads"], c["dim"], c["page"], c["layers"]
    _, tables = _tables_of(st)
    seq, pos = _tokens_of(st)
    cos, sin = st["rope"][pos][:, None].chunk(2, -1)
    q = _rotate(st["q"].float(), cos, sin).bfloat16()
    _write(st["pool"], tables, st["layer"], (L, Hk, D, P), seq, pos, _rotate(st["k"].float(), cos, sin), st["v"].float())
    # read back the cells that hold the tokens
    cells = st["pool"].view(-1, L, Hk, P // CELL, _cell_bytes(D))[tables[seq, pos // P].long(), st["layer"], :, (pos % P) // CELL]
    slot, off, kv = pos % CELL, _offsets(D), []
    for o, p in ((off[0], off[2]), (off[1], off[3])):
        by = torch.gather(cells, 2, o[slot][:, None].expand(-1, Hk, -1))
        u = torch.stack([by & 15, by >> 4], -1).flatten(-2).float()
        par = torch.gather(cells, 2, p[slot].flatten(1)[:, None].expand(-1, Hk, -1)).view(torch.float16).float().view(len(pos), Hk, -1, 2)
        kv.append(((u.view(len(pos), Hk, -1, GROUP) - 8.0) * par[..., 0:1] + par[..., 1:2]).view(len(pos), Hk, D).bfloat16())
    return {"q": q, "k": kv[0], "v": kv[1]}


def _plain_fork(st):
    c = st["case"]
    P, L, Hk, D = c["page"], c["layers"], c["kv_heads"], c["dim"]
    info, lens, refs, tables = _views(st)
    src, dst = st["src"].long(), st["dst"].long()
    # free
    old = tables[dst].flatten().long()
    refs.index_add_(0, old.clamp(min=0), -(old >= 0).int())
    tables[dst] = -1
    lens[dst] = 0
    # fork: the full pages shared, the partial page's cells copied into the lowest free pages in order
    full, rem = lens[src] // P, lens[src] % P
    col = torch.arange(tables.shape[1], device=DEV)
    shared = torch.where(col[None] < full[:, None], tables[src], torch.full_like(tables[src], -1))
    flat = shared.flatten().long()
    refs.index_add_(0, flat.clamp(min=0), (flat >= 0).int())
    tables[dst] = shared
    part = torch.nonzero(rem > 0).flatten()
    got = torch.nonzero(refs == 0).flatten()[:part.numel()]
    frm = tables[src[part], full[part].long()].long()
    pool = st["pool"].view(-1, L, Hk, P // CELL, _cell_bytes(D))
    used = torch.arange(P // CELL, device=DEV)[None] * CELL < rem[part][:, None]
    pool[got] = torch.where(used[:, None, None, :, None], pool[frm], pool[got])
    tables[dst[part], full[part].long()] = got.int()
    refs[got] = 1
    lens[dst] = lens[src]
    # reserve one token each
    grow = torch.nonzero(lens[dst] % P == 0).flatten()
    got = torch.nonzero(refs == 0).flatten()[:grow.numel()]
    tables[dst[grow], (lens[dst[grow]] // P).long()] = got.int()
    refs[got] = 1
    lens[dst] += 1
    info[0] = (refs == 0).sum()
    info[1] = 0
    return {"pool": st["pool"], "book": st["book"]}


def _plain_compact(st):
    st["book"].copy_(st["saved"])
    info, lens, refs, tables = _views(st)
    n = int((refs > 0).sum())
    holes = torch.nonzero(refs[:n] == 0).flatten()
    movers = n + torch.nonzero(refs[n:] > 0).flatten()
    st["pool"][holes] = st["pool"][movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    to = torch.arange(refs.numel(), device=DEV, dtype=torch.int32)
    to[movers] = holes.int()
    tables.copy_(torch.where(tables >= 0, to[tables.clamp(min=0).long()], tables))
    info[2] = holes.numel()
    return {"pool": st["pool"], "book": st["book"]}


_OWN = {"attention": _own_attention, "append": _own_append, "fork": _own_fork, "compact": _own_compact}
_PLAIN = {"attention": _plain_attention, "append": _plain_append, "fork": _plain_fork, "compact": _plain_compact}


# --- the definition in 64 bits ----------------------------------------------------------

def _stored(pool, pages, layer, case, h, n):
    """K, V (fp64 [n][D]) of one kv head of a sequence, straight from the format's definition."""
    D, P, L, H = case["dim"], case["page"], case["layers"], case["kv_heads"]
    G, cb = D // 64, _cell_bytes(D)
    t = torch.arange(n, device=DEV)
    base = (((pages[t // P].long() * L + layer) * H + h) * (P // 16) + (t % P) // 16) * cb
    flat, w, ch = pool.view(-1), (t % 16)[:, None], torch.arange(D, device=DEV)[None]
    grp, x = ch // 64, ch % 64
    # K: a row of D/2 bytes per token, in pieces of 16 channels of each group; two channels to a byte, low bits first
    kb = w * (D // 2) + (x // 16) * 8 * G + grp * 8 + (x % 16) // 2
    # V: 16-byte pieces of 8 channels x (tokens 2j, 2j+1, 2j+8, 2j+9); four channels of a token in two bytes
    vb = 8 * D + grp * 512 + ((x // 8) * 4 + (w % 8) // 2) * 16 + (w // 8) * 8 + ((x // 4) % 2) * 4 + (w % 2) * 2 + (x % 4) // 2
    half = pool.view(torch.float16).view(-1)
    kp = (base[:, None] + 16 * D + (w * G + grp) * 4) // 2
    vp = (base[:, None] + 16 * D + 64 * G + ((w // 2) * G + grp) * 8 + (w % 2) * 2) // 2
    out = []
    for at, s, mid in ((kb, kp, kp + 1), (vb, vp, vp + 2)):
        code = (flat[base[:, None] + at].to(torch.int32) >> (4 * (ch % 2))) & 15
        out.append(half[mid].double() + half[s].double() * (code.double() - 8))
    return out


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None
    st = prepare(case, seed)
    H, Hk, D, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    lens, new = _ints(case["lens"]), _ints(case["new"])
    n = len(lens)
    if case["op"] == "append":
        pos = torch.cat([torch.arange(a - b, a, device=DEV) for a, b in zip(lens, new)])
        angle = st["rope"][pos].double()[:, None]
        half = D // 2
        def turned(x):
            x = x.double()
            y = torch.empty_like(x)
            y[..., :half] = x[..., :half] * angle[..., :half] - x[..., half:] * angle[..., half:]
            y[..., half:] = x[..., half:] * angle[..., :half] + x[..., :half] * angle[..., half:]
            return y
        res = {"q": turned(st["q"])}
        for name, x in (("k", turned(st["k"])), ("v", st["v"].double())):
            x = x.reshape(x.shape[0], Hk, D // 64, 64)
            least = x.min(-1, keepdim=True).values
            s = ((x.max(-1, keepdim=True).values - least) / 15).bfloat16().half().double()
            mid = (least + 8 * s).half().double()
            res[name] = (mid + s * torch.clamp(torch.round((x - mid) / s), -8, 7)).reshape(-1, Hk, D)
        return res
    out = torch.zeros(sum(new), H, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(sum(new), H, dtype=torch.float64, device=DEV)
    max_pages = max(-(-x // P) for x in lens) + 1
    tables = st["book"][16 + _pad4(n) + _pad4(st["pool"].shape[0]):][:n * max_pages].view(n, max_pages)
    at = 0
    for s in range(n):
        q = st["q"][at:at + new[s]].double()
        hidden = torch.arange(lens[s], device=DEV)[None] > torch.arange(lens[s] - new[s], lens[s], device=DEV)[:, None]
        for h in range(Hk):
            K, V = _stored(st["pool"], tables[s], st["layer"], case, h, lens[s])
            for j in range(h * (H // Hk), (h + 1) * (H // Hk)):
                x = (q[:, j] @ K.T / D ** 0.5).masked_fill(hidden, float("-inf"))
                lse[at:at + new[s], j] = torch.logsumexp(x, -1)
                out[at:at + new[s], j] = torch.softmax(x, -1) @ V
        at += new[s]
    return {"out": out, "lse": lse}
