"""One decoder layer on the library's calls: the 4-bit products, and between
them rotary positions, the paged cache and the attention over it.

    qkv   = W_qkv norm(x)                 w4_gemv
    cache <- rotate(k), v; q <- rotate(q) w4_kv_append   (one launch)
    a     = attention(q, cache)           w4_paged_attn
    x     = x + W_o a                     w4_gemv
    x     = x + W_down swiglu(W_gate_up norm(x))   w4_gemv_swiglu, w4_gemv

A prompt goes through in chunks of up to 8 tokens (the token counts of the
products), then tokens are decoded one at a time, or several draft tokens at
once as a speculative step would; the rows come out the same up to the
rounding of the sums.  Norms and residual sums are torch operations: the
library has none.  Weights are synthetic, in the shapes of the library's
workloads.

    python examples/decode_layer.py [--shape 0.5b|7b] [--cache bf16|int8|int4]
                                    [--seqs 4] [--prompt 100] [--steps 16] [--draft 1]
"""
from __future__ import annotations

import argparse
import os
import sys
import time
from dataclasses import dataclass

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from int4_weight_only_w4_gb300 import synthetic, w4  # noqa: E402


@dataclass
class Shape:
    hidden: int
    inner: int
    q_heads: int
    kv_heads: int
    head_dim: int


SHAPES = {"0.5b": Shape(896, 4864, 14, 2, 64), "7b": Shape(3584, 18944, 28, 4, 128)}
FORMATS = {"bf16": w4.KV_BF16, "int8": w4.KV_INT8, "int4": w4.KV_INT4}


def _canonical(name: str, K: int, N: int, seed: int):
    """A synthetic weight with entries of about 1 / sqrt(K), on the device."""
    top = 0.35 / K ** 0.5
    qw, sc, zp = synthetic.make_weights(name, K, N, seed, (0.5 * top, top))
    return (torch.from_numpy(qw.view(np.int32)).cuda(), torch.from_numpy(sc.view(np.int16)).cuda(),
            torch.from_numpy(zp).cuda())


def _norm(x: torch.Tensor) -> torch.Tensor:
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Layer:
    """The layer's weights, its rotation table and its cache with a block table
    of `seqs` sequences of up to `longest` tokens."""

    def __init__(self, shape: Shape, fmt: str, seqs: int, longest: int, page_tokens: int = 16,
                 seed: int = 0):
        s = self.shape = shape
        qkv = (s.q_heads + 2 * s.kv_heads) * s.head_dim
        self.qkv = w4.pack(*_canonical("layer.qkv", s.hidden, qkv, seed), s.hidden, qkv)
        self.o = w4.pack(*_canonical("layer.o", s.q_heads * s.head_dim, s.hidden, seed),
                         s.q_heads * s.head_dim, s.hidden)
        self.gate_up = w4.pack_swiglu(*_canonical("layer.gate_up", s.hidden, 2 * s.inner, seed),
                                      s.hidden, s.inner)
        self.down = w4.pack(*_canonical("layer.down", s.inner, s.hidden, seed), s.inner, s.hidden)
        self.rope = w4.RopeTable.make(longest, s.head_dim, base=1e6)
        pages = -(-longest // page_tokens)
        self.cache = w4.PagedCache.make(seqs * pages, FORMATS[fmt], s.kv_heads, s.head_dim,
                                        page_tokens)
        gen = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(seqs * pages, generator=gen).view(seqs, pages)
        self.table = self.table.to(torch.int32).cuda()

    def _product(self, weight, x: torch.Tensor) -> torch.Tensor:
        """weight.gemv over any number of rows, 8 at a time."""
        return torch.cat([weight.gemv(part.contiguous()) for part in x.split(w4.MAX_TOKENS)])

    def step(self, x: torch.Tensor, lens: torch.Tensor) -> torch.Tensor:
        """x [seqs * tokens, hidden] bfloat16, `tokens` new ones (1..8) of every
        sequence; lens int32 [seqs]: their lengths with these tokens."""
        s, B = self.shape, lens.numel()
        M = x.shape[0] // B
        rows = self._product(self.qkv, _norm(x)).view(B * M, -1, s.head_dim)
        q, k, v = rows.split([s.q_heads, s.kv_heads, s.kv_heads], 1)
        positions = (lens[:, None] - M + torch.arange(M, device=lens.device, dtype=torch.int32))
        self.cache.append(k, v, positions.reshape(-1), self.table, q=q, q_out=q, rope=self.rope)
        a, _ = self.cache.attend(q, lens, self.table)
        x = x + self._product(self.o, a.view(B * M, -1))
        return x + self._product(self.down, self._product(self.gate_up, _norm(x)))


def run(shape: str = "0.5b", fmt: str = "int4", seqs: int = 4, prompt: int = 100, steps: int = 16,
        draft: int = 1, seed: int = 0):
    """The layer over a prompt and `steps` more tokens, `draft` at a time.
    Returns its outputs [seqs, prompt + steps, hidden] and the seconds of a step."""
    s = SHAPES[shape]
    total = prompt + steps
    layer = Layer(s, fmt, seqs, total, seed=seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(seqs, total, s.hidden, generator=gen, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(x)
    at, took = 0, 0.0
    while at < total:
        M = min(w4.MAX_TOKENS, prompt - at) if at < prompt else min(draft, total - at)
        lens = torch.full((seqs,), at + M, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        began = time.perf_counter()
        out[:, at:at + M] = layer.step(x[:, at:at + M].reshape(seqs * M, -1),
                                       lens).view(seqs, M, -1)
        torch.cuda.synchronize()
        took = time.perf_counter() - began
        at += M
    layer.cache.check()
    return out, took


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--shape", choices=SHAPES, default="0.5b")
    p.add_argument("--cache", choices=FORMATS, default="int4")
    p.add_argument("--seqs", type=int, default=4)
    p.add_argument("--prompt", type=int, default=100)
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--draft", type=int, default=1)
    a = p.parse_args()
    exact, _ = run(a.shape, "bf16", a.seqs, a.prompt, a.steps, 1)
    out, took = run(a.shape, a.cache, a.seqs, a.prompt, a.steps, a.draft)
    off = (out.float() - exact.float()).norm() / exact.float().norm()
    print(f"{a.shape} layer, {a.seqs} sequences, {a.prompt} + {a.steps} tokens, {a.cache} cache, "
          f"{a.draft} a step: {1e6 * took:.0f} us the last step, "
          f"{off:.2e} from single steps over a bf16 cache")


if __name__ == "__main__":
    main()
