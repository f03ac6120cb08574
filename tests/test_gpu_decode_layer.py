"""The decoder-layer example: its outputs with every cache format and step
size against the same layer in plain fp32 torch over dequantised weights, with
keys and values as a cache of that format holds them."""
import importlib.util
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

from tests import kv_testutil as kv  # noqa: E402

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = mod
    spec.loader.exec_module(mod)
    return mod


def plain(ex, shape, fmt, seqs, total, seed=0):
    """fp32; activations are rounded to bfloat16 where the layer's are."""
    from int4_weight_only_w4_gb300 import synthetic
    s = ex.SHAPES[shape]
    r = lambda t: t.to(torch.bfloat16).float()  # noqa: E731

    def weight(name, K, N):
        top = 0.35 / K ** 0.5
        qw, sc, zp = synthetic.make_weights(name, K, N, seed, (0.5 * top, top))
        q = (qw[..., None] >> (4 * np.arange(8, dtype=np.uint32))) & 15
        q = q.reshape(N, K // 128, 128).astype(np.float32) - zp[..., None].astype(np.float32)
        w = q * sc.view(np.float16)[..., None].astype(np.float32)
        return torch.from_numpy(w.reshape(N, K)).cuda()

    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(seqs, total, s.hidden, generator=gen, device="cuda").to(torch.bfloat16).float()
    norm = lambda t: r(t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6))  # noqa: E731
    D, H, HQ = s.head_dim, s.kv_heads, s.q_heads
    rows = r(norm(x) @ weight("layer.qkv", s.hidden, (HQ + 2 * H) * D).T)
    q, k, v = rows.view(seqs, total, -1, D).split([HQ, H, H], 2)
    f = 1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
    ang = torch.arange(total, device="cuda", dtype=torch.float64)[:, None] * f
    c, sn = ang.cos().float()[:, None], ang.sin().float()[:, None]
    turn = lambda t: torch.cat([t[..., :D // 2] * c - t[..., D // 2:] * sn,  # noqa: E731
                                t[..., D // 2:] * c + t[..., :D // 2] * sn], -1)
    q, k = r(turn(q)), turn(k)
    k, v = (torch.from_numpy(kv.held(t.cpu().numpy(), fmt)).cuda() for t in (k, v))
    k, v = (t.repeat_interleave(HQ // H, 2) for t in (k, v))
    p = torch.einsum("bihd,bjhd->bhij", q, k) / D ** 0.5
    p = p.masked_fill(torch.ones(total, total, device="cuda").triu(1).bool(), -torch.inf).softmax(-1)
    a = r(torch.einsum("bhij,bjhd->bihd", p, v)).reshape(seqs, total, -1)
    x = r(x + r(a @ weight("layer.o", HQ * D, s.hidden).T))
    gu = norm(x) @ weight("layer.gate_up", s.hidden, 2 * s.inner).T
    g, u = gu.split(s.inner, -1)
    return r(x + r(r(g * torch.sigmoid(g) * u) @ weight("layer.down", s.inner, s.hidden).T))


# Activations are rounded to bfloat16 in about ten places (2^-9 relative each,
# in the root mean square 2^-9.8, over at most 10: sqrt(10) * 2^-9.8 = 0.0036).
# The two sides' qkv products round differently in some 5 % of the values, by
# 2^-8; where that moves a value over a code's border, a whole step of about
# 6 / 15 of the deviation changes in 4 bits: in 1 % of these, together
# sqrt(0.05 * 0.01) * 0.4 = 0.009 of keys and of values; in 8 bits it is 0.002.
LIMIT = {"bf16": 0.01, "int8": 0.012, "int4": 0.03}


@pytest.mark.parametrize("fmt", list(LIMIT))
@pytest.mark.parametrize("shape,seqs,prompt,steps,draft", [
    ("0.5b", 3, 37, 5, 1), ("0.5b", 1, 16, 9, 4), ("7b", 2, 21, 8, 8)])
def test_layer(example, fmt, shape, seqs, prompt, steps, draft):
    out, _ = example.run(shape, fmt, seqs, prompt, steps, draft)
    ref = plain(example, shape, fmt, seqs, prompt + steps)
    err = (out.float() - ref).norm() / ref.norm()
    assert err <= LIMIT[fmt], float(err)
