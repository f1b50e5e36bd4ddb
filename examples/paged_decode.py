"""A decode loop over pruned linears and a paged KV cache, in 4 or 8 bits.

A few decoder layers with random weights: the linears are pruned to 2:4 and run as the
bitmask SpMV, the attention between qkv and o reads the paged cache. A prompt goes in
eight tokens at a time (the largest batch of the SpMV), is forked into several
continuations that share its full pages, and these are decoded together; then all but
one are dropped and the pool is compacted. The "sampling" takes the next input from the
last hidden state, so no vocabulary is needed. With the 8-bit cache and --pages a step
attends only the pages whose keys can have the largest scores.

    python examples/paged_decode.py [--layers 2 --hidden 1024 --prompt 100 --steps 20 --bits 8 --pages 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_decoding_gb300 as nm  # noqa: E402


def rope_table(positions: int, dim: int, theta: float = 500000.0, device="cuda") -> torch.Tensor:
    """cos and sin of every position's angles, fp32 [positions][dim]."""
    inv = theta ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=device) / dim)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class Decoder:
    """Decoder layers over one cache. ``step`` runs all of them on up to eight tokens."""

    def __init__(self, layers=2, hidden=1024, heads=8, kv_heads=2, dim=128, ffn=2048, sequences=4, tokens=512, page=16,
                 seed=0, device="cuda", bits=4, pages=0):
        if pages < 0 or (pages and bits != 8):
            raise ValueError("pages are selected in the 8-bit cache, at least one")
        self.heads, self.kv_heads, self.dim, self.pages = heads, kv_heads, dim, pages
        max_pages = -(-tokens // page)
        self.cache = (nm.Kv8Cache if bits == 8 else nm.Kv4Cache)(sequences * max_pages, page, layers, kv_heads, dim, sequences, max_pages, device=device)
        self.rope = rope_table(tokens, dim, device=device)
        g = torch.Generator(device=device).manual_seed(seed)

        def pruned(rows, cols):
            W = (torch.randn(rows, cols, generator=g, device=device) * cols ** -0.5).bfloat16()
            return nm.select(W, torch.ones(cols, device=device), 2, 4)

        self.layers = []
        for _ in range(layers):
            self.layers.append({
                "qkv": nm.pack(pruned((heads + 2 * kv_heads) * dim, hidden), 2, 4),
                "o": nm.pack(pruned(hidden, heads * dim), 2, 4),
                "gate_up": nm.pack_swiglu(pruned(ffn, hidden), pruned(ffn, hidden), 2, 4),
                "down": nm.pack(pruned(hidden, ffn), 2, 4),
            })

    @staticmethod
    def norm(x: torch.Tensor) -> torch.Tensor:
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def step(self, x: torch.Tensor, seqs: torch.Tensor, starts=None, trace=None) -> torch.Tensor:
        """x bf16 [tokens][hidden] -> the layers' output. The tokens are the next of the listed
        sequences: one each, or starts[i] .. starts[i + 1] of sequence i. ``trace`` (a list) gets
        each layer's q, k, v before the rotation and the attention's result."""
        c, D = self.cache, self.dim
        c.reserve(seqs, starts)  # once for all layers
        for i, w in enumerate(self.layers):
            q, k, v = nm.spmv_qkv(*w["qkv"], self.norm(x), self.heads * D, self.kv_heads * D)
            if trace is not None:
                trace.append([q.clone(), k.clone(), v.clone()])
            c.append(i, k, v, q=q, rope=self.rope, seqs=seqs, starts=starts, q_out=q)
            # of a single page the token's own, else the first one too
            part = {"pages": c.select(i, q, self.pages, seqs=seqs, starts=starts, first=min(1, self.pages - 1))} if self.pages else {}
            a = c.attention(i, q, seqs=seqs, starts=starts, max_new=1 if starts is None else x.shape[0], **part)
            if trace is not None:
                trace[-1].append(a)
            x = x + nm.spmv(*w["o"], a)
            x = x + nm.spmv(*w["down"], nm.spmv_swiglu(*w["gate_up"], self.norm(x)))
        return x


def run(decoder: Decoder, prompt: torch.Tensor, branches: int, steps: int):
    """The prompt into sequence 0, `branches` sequences decoded from it `steps` times; the first is
    kept. Returns the last hidden states of all branches, step by step."""
    c = decoder.cache

    def ids(*x):
        return torch.tensor(x, dtype=torch.int32, device=c.device)

    first, x = ids(0), None
    for a in range(0, prompt.shape[0], 8):
        chunk = prompt[a:a + 8]
        x = decoder.step(chunk, first, starts=ids(0, chunk.shape[0]))
    others, every = ids(*range(1, branches)), ids(*range(branches))
    if branches > 1:
        c.fork(first.repeat(branches - 1), others)
    x = x[-1:].repeat(branches, 1) * torch.linspace(1, 2, branches, device=c.device, dtype=x.dtype)[:, None]
    out = []
    for _ in range(steps):
        x = decoder.step(decoder.norm(x), every)
        out.append(x)
    if branches > 1:
        c.free(others)
    c.compact()
    return out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("layers", 2), ("hidden", 1024), ("prompt", 100), ("branches", 3), ("steps", 20), ("bits", 4), ("pages", 0)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    nm.init()
    d = Decoder(layers=a.layers, hidden=a.hidden, sequences=max(a.branches, 1), tokens=a.prompt + a.steps + 1,
                bits=a.bits, pages=a.pages)
    prompt = torch.randn(a.prompt, a.hidden, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    out = run(d, prompt, a.branches, a.steps)
    free, refused, moved = d.cache.info.tolist()[:3]
    assert refused == 0 and nm.device_status() == nm.NM_OK
    print(f"{a.prompt} prompt tokens, {a.branches} branches x {a.steps} steps; last state norms "
          f"{[round(float(v), 3) for v in out[-1].float().norm(dim=-1)]}; {free} of {d.cache.n_pages} pages free, {moved} moved")


if __name__ == "__main__":
    main()
