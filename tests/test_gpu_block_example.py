"""examples/decoder_block.py, small, against the same block in float64: the oracle's dequantised weights, the oracle's
cache and attention. Prompts of different lengths, then decode steps that fill cache blocks.

Tolerance: the linears' own bound is 2e-3 of sum |x||w| (oracle.TOL_REL), about 2e-3 sqrt(K) of an output's size at
worst and a few 1e-4 of it in the norm; with the seven fp16 roundings of a block (2^-11 each) and the cache's codes
moving by a step where a key's last fp16 bit does, 1e-2 in the norm leaves a factor of several."""
import importlib.util
import os

import numpy as np
import pytest

import oracle
from oracle import block as ob

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    import torch
    assert torch.cuda.is_available(), "GPU tests need an MI355X; none is visible"
    spec = importlib.util.spec_from_file_location("decoder_block", os.path.join(ROOT, "examples", "decoder_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt,heads,kv_heads,D", [("int8", 8, 2, 64), ("e4m3", 4, 4, 128)])
def test_block_against_float64(ex, fmt, heads, kv_heads, D):
    import torch
    hidden, inner, theta = heads * D, 768, 10000.0
    w = ex.random_weights(hidden, heads, kv_heads, D, inner, seed=3)
    rope = ex.bk.Rope(D, 200, theta=theta)
    layer = ex.DecoderBlock(w, heads, kv_heads, D, rope, rho=0.01)
    ref = {n: oracle.dequant(oracle.pack(w[n].cpu().numpy(), 128, 0.01)).astype(np.float64)
           for n in ("q", "k", "v", "o", "gate", "up", "down")}
    norms = {n: w[n].cpu().numpy().astype(np.float64) for n in ("norm_attn", "norm_mlp", "norm_next")}
    seqs = ex.Sequences(3, 200, kv_heads, D, fmt)
    table = seqs.table.cpu().numpy()
    cache = ob.Cache(table.size, 3, kv_heads, D, fmt)
    f, _ = ob.frequencies(D, theta)
    lens = [0, 0, 0]

    def norm(x, g):
        return x / np.sqrt((x * x).mean(1, keepdims=True) + 1e-6) * g

    def block64(r, new):
        h = norm(r, norms["norm_attn"])
        q, k, v = ((h @ ref[n].T).reshape(len(r), -1, D) for n in ("q", "k", "v"))
        pos = np.concatenate([np.arange(L, L + n) for L, n in zip(lens, new)])
        q, k = ob.rope(q, pos, f), ob.rope(k, pos, f)
        a, at = np.zeros((len(r), heads, D)), 0
        for s, n in enumerate(new):
            L = lens[s] + n
            cache.put(L, list(table[s]), s, k[at:at + n].astype(np.float16), v[at:at + n].astype(np.float16))
            for h_ in range(heads):
                kk, vv = cache.read(L, list(table[s]), s, h_ * kv_heads // heads)
                for i in range(n):
                    a[at + i, h_] = ob.attend(q[at + i, h_], kk, vv, L - n + i + 1, D ** -0.5)[0]
            at += n
        r = r + a.reshape(len(r), -1) @ ref["o"].T
        h = norm(r, norms["norm_mlp"])
        g, u = h @ ref["gate"].T, h @ ref["up"].T
        r = r + (g / (1 + np.exp(-g)) * u) @ ref["down"].T
        return r, norm(r, norms["norm_next"])

    g = np.random.default_rng(1)
    for new in ([63, 70, 5], [1, 1, 1], [1, 1, 1], [20, 58, 1]):
        r = g.standard_normal((sum(new), hidden)).astype(np.float32)
        rd = torch.from_numpy(r).cuda()
        r2, h2 = layer(rd, layer.first_norm(rd), seqs.cache, seqs.batch(new))
        want_r, want_h = block64(r.astype(np.float64), new)
        lens = [L + n for L, n in zip(lens, new)]
        for got, want, what in ((r2, want_r, "residual"), (h2, want_h, "normed")):
            err = np.linalg.norm(got.cpu().numpy().astype(np.float64) - want) / np.linalg.norm(want)
            assert err <= 1e-2, (what, new, err)


def test_example_runs(ex, capsys, monkeypatch):
    import sys
    monkeypatch.setattr(sys, "argv", ["decoder_block.py", "--hidden", "512", "--heads", "8", "--kv-heads", "2",
                                      "--inner", "1024", "--sequences", "4", "--prompt", "150", "--steps", "70"])
    ex.main()
    assert "us a step" in capsys.readouterr().out
