"""The way out of a model, as it is measured: the last norm with its residual and an output in 8 bits, the product of
8-bit rows with 8-bit weights (the head's, or any layer that is not held in 4 bits), and the sampling of a token.

`own` false computes the plain form: elementary torch operations in 32 bits (64 for the sampler's weights), rounded
once at the end. `own` true makes the framework's calls (bit_gemm_amd.block, bit_gemm_amd.head). exact() is the
definition in 64 bits, written apart.

8-bit rows. x [rows, K] is held as codes e4m3 [rows, Kp], Kp = 128 ceil(K / 128), zero past K, and a scale for each
block of 128, a power of two (e8m0) [rows, Kp / 128]: the smallest 2^e with max |x| <= 448 2^e, 1 where the block is
all zero; code = x / 2^e, rounded to nearest even. Weights [N, K] are held in the same way.

Sampling. Weights are whole numbers w = rint(2^40 exp((l - max) / temperature)); tokens are ordered by logit, the
lower index first among equals. Kept are the first top_k; of those the ones with w >= min_p 2^40; and the ones with
less than top_p T before them, T the sum of the first top_k. The token is the first by index whose running sum of kept
weights passes u times their sum; its log-probability is ln(w / sum). Temperature 0 takes the first largest logit.
"""
import math
import random

import torch

own = False

BLOCK = 128                     # elements that share a scale
E4M3_MAX = 448.0
EPS = 1e-6
ONE = 1 << 40                   # weight of the largest logit


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # before the head of a 4096-wide model, one token for each of 16 running sequences, residual in float16
        dict(name="norm, 16 tokens", op="norm", tokens=16, width=4096, post=False, gate="none", resid="half",
             alpha=1.0, beta=1.0, offset=0.0),
        # a prompt on the 8192-wide block, residual in float32, a gate for each token and channel, scaled branch
        dict(name="norm, 4096 tokens", op="norm", tokens=4096, width=8192, post=True, gate="token", resid="float",
             alpha=1.0, beta=0.22, offset=1.0),
        # one conversation, a projection of the 4096-wide block: latency and the reading of 17 MB
        dict(name="linear, 1 token", op="linear", tokens=1, out=4096, width=4096, src="codes"),
        # 16 sequences, the 11008 x 4096 layer, rows that come in float16 and are coded on the way
        dict(name="linear, 16 tokens", op="linear", tokens=16, out=11008, width=4096, src="half"),
        # the head over a large vocabulary at 16 sequences: a stream of half a gigabyte
        dict(name="head, 16 tokens", op="linear", tokens=16, out=131072, width=4096, src="codes"),
        # a ragged batch on odd sizes: the last block of the rows is partly empty
        dict(name="linear, 333 tokens", op="linear", tokens=333, out=10007, width=2501, src="codes"),
        # a piece of a prompt on a long inner side (few output tiles)
        dict(name="linear, 512 tokens", op="linear", tokens=512, out=4096, width=14336, src="half"),
        # a prompt of 2048 tokens on the 28672 x 8192 layer
        dict(name="linear, 2048 tokens", op="linear", tokens=2048, out=28672, width=8192, src="codes"),
        # one conversation: latency
        dict(name="sample, 1 x 32000", op="sample", rows=1, vocab=32000, dtype="half", temperature=0.8, top_k=50,
             top_p=0.95, min_p=0.0, mixed=False, masked=0.0),
        # 16 sequences over a large vocabulary, nucleus alone
        dict(name="sample, 16 x 131072", op="sample", rows=16, vocab=131072, dtype="half", temperature=0.7, top_k=0,
             top_p=0.9, min_p=0.0, mixed=False, masked=0.0),
        # 64 sequences whose requests each bring their own settings, greedy ones among them
        dict(name="sample, 64 x 131072", op="sample", rows=64, vocab=131072, dtype="half", temperature=1.0, top_k=200,
             top_p=0.9, min_p=0.02, mixed=True, masked=0.0),
        # drawing many candidates from the whole distribution, float32 logits, odd vocabulary, a grammar's mask
        dict(name="sample, 333 x 50257", op="sample", rows=333, vocab=50257, dtype="float", temperature=1.0, top_k=0,
             top_p=1.0, min_p=0.0, mixed=False, masked=0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "sample", "sample"])
    if op == "norm":
        return dict(op=op, tokens=_log(rng, 1, 4096),
                    width=rng.choice([1024, 2048, 4096, 5120, 8192, 2 * rng.randint(100, 4000) + 1]),
                    post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token"]),
                    resid=rng.choice(["half", "float"]), alpha=rng.choice([1.0, 0.5]),
                    beta=rng.choice([1.0, 0.22, 1.4]), offset=rng.choice([0.0, 1.0]))
    if op == "linear":
        tokens = _log(rng, 1, 2048)
        out, width = _log(rng, 100, 32768), _log(rng, 100, 16384)
        if rng.random() < 0.6:          # the sizes of most layers
            out, width = 128 * max(1, out // 128), 128 * max(1, width // 128)
        return dict(op=op, tokens=tokens, out=out, width=width, src=rng.choice(["codes", "half"]))
    rows = _log(rng, 1, 333)
    return dict(op=op, rows=rows, vocab=_log(rng, 100, min(200000, (1 << 24) // rows)),
                dtype=rng.choice(["half", "float"]), temperature=rng.choice([0.3, 0.7, 1.0, 1.5]),
                top_k=rng.choice([0, 0, _log(rng, 4, 1000)]), top_p=rng.choice([1.0, 0.95, 0.9, 0.5]),
                min_p=rng.choice([0.0, 0.0, 0.05, 0.2]), mixed=rng.random() < 0.3,
                masked=rng.choice([0.0, 0.0, 0.5, 0.99]))


def _up(k):
    return (k + BLOCK - 1) // BLOCK * BLOCK


def work(case):
    if case["op"] == "norm":
        n, Kp = case["tokens"] * case["width"], _up(case["width"])
        r = 2 if case["resid"] == "half" else 4
        gate = {"none": 0, "channel": 2 * case["width"], "token": 2 * n}[case["gate"]]
        return {"bytes": n * (2 + 2 * r) + gate + 2 * case["width"] * (2 if case["post"] else 1)
                + case["tokens"] * (Kp + Kp // BLOCK), "flops": 10 * n}
    if case["op"] == "linear":
        M, N, K = case["tokens"], case["out"], case["width"]
        row = _up(K) + _up(K) // BLOCK
        return {"bytes": N * row + 2 * M * N + M * row + (2 * M * K if case["src"] == "half" else 0),
                "flops": 2 * M * N * K}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (2 if case["dtype"] == "half" else 4) + case["rows"] * 28, "flops": 10 * n}


# ---------------------------------------------------------------------------------------------------- inputs
def _normal(shape, g, hot=0):
    """Activations in float16: normal, some channels of the last axis eight times as large."""
    x = torch.randn(shape, generator=g, device="cuda")
    if hot:
        x[..., torch.randperm(shape[-1], generator=g, device="cuda")[:hot]] *= 8.0
    return x.half()


def _coded(x):
    """Codes and scales of the rows x [rows, K] (float16 or float32)."""
    rows, K = x.shape
    x = torch.nn.functional.pad(x.float(), (0, _up(K) - K)).view(rows, -1, BLOCK)
    top = x.abs().amax(-1)
    m, e = torch.frexp(top / E4M3_MAX)          # top / 448 = m 2^e, 0.5 <= m < 1; a power of two is its own
    e = torch.where(top > 0, torch.where(m == 0.5, e - 1, e), torch.zeros_like(e))
    c = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn).view(rows, -1)
    return c, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _weights(case, g):
    """Weights [out, width] in float16, of the size a trained layer has, with some large columns and rows."""
    W = torch.randn((case["out"], case["width"]), generator=g, device="cuda", dtype=torch.float16)
    W *= 0.02
    W[torch.randperm(case["out"], generator=g, device="cuda")[:case["out"] // 64]] *= 4.0
    return W


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "norm":
        M, H = case["tokens"], case["width"]
        dt = torch.float16 if case["resid"] == "half" else torch.float32
        st["y"] = _normal((M, H), g, 4)
        st["r"] = (torch.randn((M, H), generator=g, device="cuda") * 3).to(dt)
        for name, on in (("w_pre", True), ("w_post", case["post"])):
            w = (1.0 - case["offset"] + 0.1 * torch.randn(H, generator=g, device="cuda")).half()
            st[name] = w if on else None
        shape = {"none": None, "channel": (1, H), "token": (M, H)}[case["gate"]]
        st["gate"] = None if shape is None else torch.rand(shape, generator=g, device="cuda").half().expand(M, H)
        return st
    if op == "linear":
        W = _weights(case, g)
        x = _normal((case["tokens"], case["width"]), g, 4)
        if case["src"] == "half":
            st["x"] = x
        else:
            st["codes"], st["scales"] = _coded(x)
        if own:
            from bit_gemm_amd import head
            st["layer"] = head.mq_pack8(W)
        else:
            parts = [_coded(w) for w in W.split(16384)]
            st["w_codes"], st["w_scales"] = (torch.cat([p[i].view(torch.uint8) for p in parts]).view(parts[0][i].dtype)
                                             for i in range(2))
        return st
    R, V = case["rows"], case["vocab"]
    # logits of a trained head: most of the vocabulary far below, some dozens of tokens likely, of any sharpness
    l = torch.randn((R, V), generator=g, device="cuda") * 2.0
    n = min(V, 48)
    likely = torch.randint(V, (R, n), generator=g, device="cuda")
    boost = torch.rand((R, n), generator=g, device="cuda") * (4.0 + 10.0 * torch.rand((R, 1), generator=g, device="cuda"))
    l.scatter_add_(1, likely, boost)
    if case["masked"]:
        l.masked_fill_(torch.rand((R, V), generator=g, device="cuda") < case["masked"], -math.inf)
        l[:, V // 2] = 1.0
    st["logits"] = l.half() if case["dtype"] == "half" else l
    st["u"] = torch.rand(R, generator=g, device="cuda")
    for name, dt in (("temperature", torch.float32), ("top_k", torch.int32), ("top_p", torch.float32), ("min_p", torch.float32)):
        st[name] = torch.full((R,), case[name], dtype=dt, device="cuda")
    if case["mixed"]:               # requests of several users: some greedy, some without one limit or another
        def some(share):
            return torch.rand(R, generator=g, device="cuda") < share
        st["temperature"] *= 0.5 + torch.rand(R, generator=g, device="cuda")
        st["temperature"][some(0.1)] = 0.0
        st["top_k"][some(0.5)] = 0
        st["top_p"][some(0.3)] = 1.0
        st["min_p"][some(0.5)] = 0.0
    return st


# ---------------------------------------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return _own[op](st, st["case"])
    return _plain[op](st, st["case"])


def _own_norm(st, case):
    from bit_gemm_amd import block
    r, codes, scales = block.mq_norm_residual_q8(st["y"], st["r"], st["w_pre"], w_post=st["w_post"], gate=st["gate"],
                                                 alpha=case["alpha"], beta=case["beta"], weight_offset=case["offset"])
    return {"r": r, "codes": codes, "scales": scales}


def _own_linear(st, case):
    from bit_gemm_amd import head
    if case["src"] == "codes":
        return {"y": head.mq_linear8(st["codes"], st["scales"], st["layer"])}
    codes, scales = head.mq_quantize8(st["x"])
    return {"codes": codes, "scales": scales, "y": head.mq_linear8(codes, scales, st["layer"])}


def _own_sample(st, case):
    from bit_gemm_amd import head
    token, logprob = head.mq_sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"],
                                    top_p=st["top_p"], min_p=st["min_p"])
    return {"token": token, "logprob": logprob}


def _plain_norm(st, case):
    y = st["y"].float()
    if st["w_post"] is not None:
        y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * (st["w_post"].float() + case["offset"])
    if st["gate"] is not None:
        y = y * st["gate"].float()
    r = st["r"].float() * case["alpha"] + y * case["beta"]
    r = r.to(st["r"].dtype)
    h = r.float()
    h = h * (h.square().mean(-1, keepdim=True) + EPS).rsqrt() * (st["w_pre"].float() + case["offset"])
    codes, scales = _coded(h)
    return {"r": r, "codes": codes, "scales": scales}


def _values(codes, scales):
    return (codes.float().view(codes.shape[0], -1, BLOCK) * scales.float()[..., None]).view(codes.shape)


def _plain_linear(st, case):
    out = {}
    codes, scales = st.get("codes"), st.get("scales")
    if case["src"] == "half":
        codes, scales = _coded(st["x"])
        out = {"codes": codes, "scales": scales}
    return out | {"y": (_values(codes, scales) @ _values(st["w_codes"], st["w_scales"]).t()).half()}


def _share(f, total):
    """floor(f total) for whole totals: f [rows] float32 in 0 .. 1 is taken to 31 bits."""
    f = (f.double() * 2.0 ** 31).floor().long()
    return f * (total >> 31) + (f * (total & (2 ** 31 - 1)) >> 31)


def _plain_sample(st, case):
    l = st["logits"].double()
    V = l.shape[1]
    top = l.amax(1)
    greedy = st["temperature"] == 0
    t = torch.where(greedy, 1.0, st["temperature"].double())
    w = (((l - top[:, None]) / t[:, None]).exp() * ONE).round().long()
    order = l.sort(dim=1, descending=True, stable=True).indices
    s = w.gather(1, order)
    k = torch.where(st["top_k"] > 0, st["top_k"], V).long()
    s *= torch.arange(V, device="cuda") < k[:, None]
    run_ = s.cumsum(1)
    need = _share(st["top_p"].clamp(0, 1), run_[:, -1]).clamp(min=1)
    keep = (run_ - s < need[:, None]) & (s.double() >= st["min_p"].double()[:, None] * ONE)
    s *= keep
    w = torch.zeros_like(w).scatter_(1, order, s)
    run_ = w.cumsum(1)
    total = run_[:, -1]
    token = (run_ <= _share(st["u"], total)[:, None]).sum(1)
    logprob = (w.gather(1, token[:, None])[:, 0].double() / total).log()
    return {"token": torch.where(greedy, order[:, 0], token).int(), "logprob": torch.where(greedy, 0.0, logprob).float()}


_own = {"norm": _own_norm, "linear": _own_linear, "sample": _own_sample}
_plain = {"norm": _plain_norm, "linear": _plain_linear, "sample": _plain_sample}


# ---------------------------------------------------------------------------------------------------- 64 bits
def _coded64(x):
    """What codes and scales stand for, codes before their rounding, in 64 bits: (x / 2^e, 2^e)."""
    rows, K = x.shape
    b = torch.zeros((rows, _up(K)), dtype=torch.float64, device="cuda")
    b[:, :K] = x
    b = b.view(rows, -1, BLOCK)
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.ceil(torch.log2(torch.where(top > 0, top, E4M3_MAX) / E4M3_MAX)), 0.0)
    return (b * torch.exp2(-e)[..., None]).view(rows, -1), torch.exp2(e)


def exact(case, seed):
    if case["op"] == "norm":
        st = prepare(case, seed)
        y = st["y"].double()
        if case["post"]:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[1] + EPS) * (st["w_post"].double() + case["offset"])
        if case["gate"] != "none":
            y = y * st["gate"].double()
        r = case["alpha"] * st["r"].double() + case["beta"] * y
        h = r / torch.sqrt((r * r).sum(-1, keepdim=True) / r.shape[1] + EPS) * (st["w_pre"].double() + case["offset"])
        codes, scales = _coded64(h)
        return {"r": r, "codes": codes, "scales": scales}
    if case["op"] == "linear":
        g = torch.Generator(device="cuda").manual_seed(seed)
        W, x = _weights(case, g), _normal((case["tokens"], case["width"]), g, 4)

        def held(m):                    # what the 8-bit rows of m stand for
            c, s = _coded64(m.double())
            return c.to(torch.float8_e4m3fn).double() * s.repeat_interleave(BLOCK, 1)
        a = held(x)
        y = torch.cat([a @ held(w).t() for w in W.split(4096)], 1)
        if case["src"] == "codes":
            return {"y": y}
        c, s = _coded64(x.double())
        return {"codes": c, "scales": s, "y": y}
    logs, st = [], prepare(case, seed)
    names = ("logits", "u", "temperature", "top_k", "top_p", "min_p")
    for l, u, t, k, p, m in zip(*(st[n].double() for n in names)):
        if t == 0:
            logs.append(torch.zeros((), dtype=torch.float64, device="cuda"))
            continue
        order = torch.argsort(l, descending=True, stable=True)
        prob = torch.softmax(l[order] / t, 0)
        if k > 0:
            prob = prob[:int(k)]
        before = (prob.cumsum(0) - prob) / prob.sum()
        n = int(((before < p) & (prob >= m * prob[0])).sum()) or 1
        kept = order[:n].sort().indices                 # back to the order of the indices
        prob = prob[:n][kept]
        c = prob.cumsum(0)
        at = int((c <= u * c[-1]).sum())
        logs.append((prob[min(at, n - 1)] / c[-1]).log())
    return {"token": None, "logprob": torch.stack(logs)}
