"""The operators between a decoder block's linears, as they are measured: rotary positions, the append to a
key/value cache of 8 bits, the attention that reads it, and the norms around a block with its gate and residual.

`own` false computes the plain form: elementary torch operations in 32 bits, rounded once at the end. `own` true
makes the framework's calls (bit_gemm_amd.block). exact() is the definition in 64 bits, written apart.

The cache. Blocks of 64 tokens; codes k [blocks, kv heads, 64, head dim] and v [blocks, kv heads, head dim, 64] with
a float32 scale for each block and kv head; a block's scale is its largest magnitude over 127 (int8) or 448 (e4m3).
The tokens of a sequence's last block, while it is not full, stay in float16 in the sequence's slot of the tails,
k [slots, kv heads, 64, head dim] and v [slots, kv heads, head dim, 64]. A block table gives a sequence's blocks.
kv_len counts a sequence's tokens with the new ones, cu_q [sequences + 1] is where each sequence's new tokens start.
"""
import math
import random

import torch

own = False

BLOCK = 64                      # tokens of a cache block
CODE_MAX = {"int8": 127.0, "e4m3": 448.0}


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # rotary positions of the 32 heads of a 4096-wide block, one token for each of 16 running sequences
        dict(name="rope, 16 tokens", op="rope", tokens=16, heads=32, dim=128, rot=128, layout="half", scaling="none",
             factor=1.0, inverse=False, start=2000),
        # a prompt, half of each head rotated, pairs side by side, positions scaled by parts for a long context
        dict(name="rope, 8192 tokens", op="rope", tokens=8192, heads=64, dim=128, rot=64, layout="interleaved",
             scaling="parts", factor=8.0, inverse=False, start=40000),
        # a decode step of 16 sequences: the joined q + k + v row of each, 32 query and 8 key/value heads; one of them
        # fills its block
        dict(name="append, 16 sequences", op="append", seqs=16, new_min=1, new_max=1, ctx_min=100, ctx_max=4110,
             align=1, heads=32, kv_heads=8, dim=128, fmt="int8", rot=128, layout="half"),
        # prompts of different lengths written in one call
        dict(name="append, 4 prompts", op="append", seqs=4, new_min=700, new_max=4096, ctx_min=0, ctx_max=0,
             align=64, heads=32, kv_heads=8, dim=128, fmt="e4m3", rot=128, layout="half"),
        # keys already rotated (rot 0), small heads, prompts that go on behind a cached prefix
        dict(name="append, heads of 64", op="append", seqs=9, new_min=33, new_max=777, ctx_min=64, ctx_max=1024,
             align=64, heads=16, kv_heads=16, dim=64, fmt="int8", rot=0, layout="half"),
        # one short conversation, one token: latency alone
        dict(name="attention, 1 x 300", op="attention", seqs=1, new_min=1, new_max=1, len_min=300, len_max=300,
             heads=32, kv_heads=8, dim=128, fmt="int8", causal=True),
        # the 4096-wide block at 16 tokens: 16 sequences of mixed lengths, as many key/value heads as query heads
        dict(name="attention, 16 x 4096", op="attention", seqs=16, new_min=1, new_max=1, len_min=500, len_max=4096,
             heads=32, kv_heads=32, dim=128, fmt="int8", causal=True),
        # long documents, 64 query heads on 8 (the 8192-wide layer)
        dict(name="attention, 2 x 65500", op="attention", seqs=2, new_min=1, new_max=1, len_min=65000, len_max=65500,
             heads=64, kv_heads=8, dim=128, fmt="e4m3", causal=True),
        # a prompt of 4096 tokens
        dict(name="attention, prompt 4096", op="attention", seqs=1, new_min=4096, new_max=4096, len_min=4096,
             len_max=4096, heads=32, kv_heads=8, dim=128, fmt="e4m3", causal=True),
        # pieces of prompts behind cached prefixes, ragged, heads of 64
        dict(name="attention, 5 pieces", op="attention", seqs=5, new_min=60, new_max=512, len_min=900, len_max=8000,
             heads=32, kv_heads=8, dim=64, fmt="int8", causal=True),
        # between attention and feed-forward of the 4096-wide block, 16 tokens, residual in float16
        dict(name="norm, 16 tokens", op="norm", tokens=16, width=4096, post=True, gate="none", resid="half",
             alpha=1.0, beta=1.0, offset=0.0),
        # a prompt on the 8192-wide block, residual in float32, a gate for each token and channel, scaled branch
        dict(name="norm, 4096 tokens", op="norm", tokens=4096, width=8192, post=True, gate="token", resid="float",
             alpha=1.0, beta=0.22, offset=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "norm"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 256])
        scaling = rng.choice(["none", "linear", "base", "parts"])
        tokens = _log(rng, 1, 8192)
        return dict(op=op, tokens=tokens, heads=min(_log(rng, 1, 64), max(1, 8192 * 8192 // (tokens * dim))),
                    dim=dim, rot=rng.choice([dim, dim // 2, 2 * rng.randint(2, dim // 2)]),
                    layout=rng.choice(["half", "interleaved"]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]), inverse=rng.random() < 0.3,
                    start=rng.randint(0, 100000))
    if op == "append":
        kv_heads, dim = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 128])
        one = rng.random() < 0.5       # single tokens, or prompts
        new = 1 if one else _log(rng, 2, 2048)
        ctx = rng.choice([0, 1]) * _log(rng, 64, 8000)
        seqs = _log(rng, 1, 128) if one else _log(rng, 1, max(1, min(16, 8192 // new)))
        return dict(op=op, seqs=seqs, new_min=(new + 1) // 2, new_max=new, ctx_min=ctx // 2, ctx_max=ctx,
                    align=1 if one else BLOCK, heads=kv_heads * rng.choice([1, 2, 4]), kv_heads=kv_heads, dim=dim,
                    fmt=rng.choice(["int8", "e4m3"]), rot=rng.choice([0, dim, dim // 2]),
                    layout=rng.choice(["half", "interleaved"]))
    if op == "attention":
        kv_heads, dim = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 128])
        group = rng.choice([1, 2, 4, 5, 8]) if kv_heads <= 8 else 1
        one = rng.random() < 0.5
        new = 1 if one else _log(rng, 2, 2048)
        length = max(new, _log(rng, 1, 32768 if one else 8192))
        seqs = _log(rng, 1, max(1, min(64, (1 << 20) // (length * kv_heads))))
        if not one:                    # keep the scores of the plain form within the listed cases'
            seqs = max(1, min(seqs, int(3e8 // (new * group * kv_heads * length))))
        return dict(op=op, seqs=seqs, new_min=(new + 1) // 2, new_max=new, len_min=(length + 1) // 2, len_max=length,
                    heads=kv_heads * group, kv_heads=kv_heads, dim=dim, fmt=rng.choice(["int8", "e4m3"]),
                    causal=rng.random() < 0.8)
    tokens = _log(rng, 1, 4096)
    return dict(op=op, tokens=tokens, width=rng.choice([1024, 2048, 4096, 5120, 8192, 2 * rng.randint(100, 4000) + 1]),
                post=rng.random() < 0.7, gate=rng.choice(["none", "channel", "token"]),
                resid=rng.choice(["half", "float"]), alpha=rng.choice([1.0, 0.5]), beta=rng.choice([1.0, 0.22, 1.4]),
                offset=rng.choice([0.0, 1.0]))


def _lens(case):
    """New tokens and whole length of every sequence: by the case alone, so that every seed has the same sizes."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    new, whole = [], []
    for _ in range(case["seqs"]):
        n = r.randint(case["new_min"], case["new_max"])
        if case["op"] == "append":
            whole.append(n + r.randint(case["ctx_min"], case["ctx_max"]) // case["align"] * case["align"])
        else:
            whole.append(max(n, r.randint(case["len_min"], case["len_max"])))
        new.append(n)
    return new, whole


def _visible(case):
    """Pairs of a new token and a cached one that it attends to."""
    new, whole = _lens(case)
    return sum(n * w - (n * (n - 1) // 2 if case["causal"] else 0) for n, w in zip(new, whole))


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n + 4 * case["tokens"] * (case["rot"] + 1),
                "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    if case["op"] == "append":
        new, whole = _lens(case)
        T, hk, D = sum(new), case["kv_heads"], case["dim"]
        b = 4 * T * hk * D + 12 * case["seqs"]
        if case["rot"]:
            b += 4 * T * case["heads"] * D + 4 * T * case["rot"]
        for n, w in zip(new, whole):
            first, done = (w - n) // BLOCK, w // BLOCK
            if done > first:                       # completed blocks: earlier tokens read, codes and scales written
                b += 4 * hk * D * ((w - n) % BLOCK) + (done - first) * hk * (2 * BLOCK * D + 8 + 4)
            b += 4 * hk * D * (w - max(w - n, done * BLOCK))     # tokens that stay open
        return {"bytes": b, "flops": (3 * T * (case["heads"] + hk) * case["rot"]) + 4 * T * hk * D}
    if case["op"] == "attention":
        new, whole = _lens(case)
        hk, D = case["kv_heads"], case["dim"]
        b = 4 * sum(new) * case["heads"] * D + 12 * case["seqs"]
        for w in whole:
            full = w // BLOCK
            b += hk * full * (2 * BLOCK * D + 8) + 4 * full + 4 * hk * D * (w - full * BLOCK)
        return {"bytes": b, "flops": 4 * D * case["heads"] * _visible(case)}
    n = case["tokens"] * case["width"]
    r = 2 if case["resid"] == "half" else 4
    gate = {"none": 0, "channel": 2 * case["width"], "token": 2 * n}[case["gate"]]
    return {"bytes": n * (4 + 2 * r) + gate + 2 * case["width"] * (2 if case["post"] else 1), "flops": 10 * n}


# ---------------------------------------------------------------------------------------------------- inputs
THETA, ORIGINAL = 500000.0, 8192


def _frequencies(rot, scaling, factor):
    """Turns of each pair a position, and the factor on cos and sin (in 64 bits, on the host)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    base, mag = THETA, 1.0
    if scaling == "base":
        base = THETA * factor ** (rot / max(1, rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":      # pairs that turn over 32 times in the original context keep their frequency, under 1 time are divided
        def at(turns):
            return rot * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(THETA))
        lo, hi = max(0.0, math.floor(at(32.0))), min(rot - 1.0, math.ceil(at(1.0)))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        f = f * (1 - ramp) + f / factor * ramp
        mag = 0.1 * math.log(factor) + 1.0
    return f, mag


def _table(rot, scaling, factor, positions):
    """cos and sin of every position and pair, [positions, rot / 2, 2] float32."""
    f, mag = _frequencies(rot, scaling, factor)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * f.cuda()[None, :]
    return torch.stack((a.cos() * mag, a.sin() * mag), -1).float()


def _normal(shape, g, hot=0):
    """Activations in float16: normal, some channels of the last axis eight times as large."""
    x = torch.randn(shape, generator=g, device="cuda")
    if hot:
        x[..., torch.randperm(shape[-1], generator=g, device="cuda")[:hot]] *= 8.0
    return x.half()


def _quantised(x, fmt):
    """Codes (int8, or e4m3 held in float8) and scales of blocks x [blocks, kv heads, :, :]."""
    amax = x.abs().amax((2, 3))
    c = x * (CODE_MAX[fmt] / amax)[..., None, None]
    c = c.round().clamp(-127, 127).to(torch.int8) if fmt == "int8" else c.clamp(-448, 448).to(torch.float8_e4m3fn)
    return c, amax / CODE_MAX[fmt]


def _cache(case, whole, g):
    """A cache that holds what a program has in it: every sequence's blocks, scattered over the pool, and its tail."""
    S, hk, D, fmt = case["seqs"], case["kv_heads"], case["dim"], case["fmt"]
    need = [(w + BLOCK - 1) // BLOCK for w in whole]
    blocks = sum(need) + 3
    ids = torch.randperm(blocks, generator=g, device="cuda").int()
    table = torch.full((S, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = ids[at:at + n]
        at += n
    st = {"block_table": table, "slots": torch.randperm(S + 2, generator=g, device="cuda")[:S].int()}
    for name, shape in (("k", (hk, BLOCK, D)), ("v", (hk, D, BLOCK))):
        hot = torch.ones((D, 1) if name == "v" else (1, D), device="cuda")
        if name == "k":
            hot[:, :2] = 6.0
        codes, scales, step = [], [], max(1, (1 << 26) // (hk * BLOCK * D))
        for b in range(0, blocks, step):
            c, s = _quantised(torch.randn((min(step, blocks - b),) + shape, generator=g, device="cuda") * hot, fmt)
            codes.append(c.view(torch.uint8))
            scales.append(s)
        codes = torch.cat(codes)
        st[name + "_codes"] = codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)
        st[name + "_scale"] = torch.cat(scales)
        st[name + "_tail"] = (torch.randn((S + 2,) + shape, generator=g, device="cuda") * hot).half()
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    if op == "rope":
        T, rot = case["tokens"], case["rot"]
        positions = case["start"] + T
        st["x"] = _normal((T, case["heads"], case["dim"]), g)
        st["pos"] = (torch.arange(T, device="cuda") + case["start"]).int()
        if own:
            from bit_gemm_amd import block
            st["rope"] = block.Rope(rot, positions, layout=case["layout"], theta=THETA, scaling=case["scaling"],
                                    factor=case["factor"], original=ORIGINAL)
        else:
            st["table"] = _table(rot, case["scaling"], case["factor"], positions)
        return st
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
    new, whole = _lens(case)
    st |= _cache(case, whole, g)
    T, hq, hk, D = sum(new), case["heads"], case["kv_heads"], case["dim"]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st["kv_len"] = torch.tensor(whole, dtype=torch.int32, device="cuda")
    st["max_new"], st["max_len"] = max(new), max(whole)
    if op == "append":          # the joined projection's output, a row for each token
        qkv = _normal((T, (hq + 2 * hk) * D), g, 8)
        q, k, v = qkv.split((hq * D, hk * D, hk * D), 1)
        st["q"], st["k"], st["v"] = q.unflatten(1, (hq, D)), k.unflatten(1, (hk, D)), v.unflatten(1, (hk, D))
    else:
        st["q"] = _normal((T, hq, D), g, 2)
    if own:
        from bit_gemm_amd import block
        st["cache"] = block.KVCache(*(st[n] for n in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail")))
        st["batch"] = block.KVBatch(st["cu_q"], st["kv_len"], st["block_table"], st["max_new"], st["max_len"],
                                    slots=st["slots"])
    if op == "append" and case["rot"]:
        if own:
            st["rope"] = block.Rope(case["rot"], max(whole), layout=case["layout"], theta=THETA)
        else:
            st["table"] = _table(case["rot"], "none", 1.0, max(whole))
    return st


# ---------------------------------------------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return _own[op](st, st["case"])
    return _plain[op](st, st["case"])


def _own_rope(st, case):
    from bit_gemm_amd import block
    return block.mq_rope(st["x"], st["rope"], st["pos"], inverse=case["inverse"])


def _own_append(st, case):
    from bit_gemm_amd import block
    q = block.mq_kv_append(st["q"], st["k"], st["v"], st["cache"], st["batch"], rope=st.get("rope"))
    return _written(st, q if case["rot"] else None)


def _own_attention(st, case):
    from bit_gemm_amd import block
    return block.mq_kv_attention(st["q"], st["cache"], st["batch"], causal=case["causal"])


def _own_norm(st, case):
    from bit_gemm_amd import block
    r, h = block.mq_norm_residual(st["y"], st["r"], st["w_pre"], w_post=st["w_post"], gate=st["gate"],
                                  alpha=case["alpha"], beta=case["beta"], weight_offset=case["offset"])
    return {"r": r, "h": h}


def _written(st, q):
    """What an append leaves: the rotated queries, where there is a rotation, and the cache."""
    out = {n: st[n] for n in ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail")}
    return out if q is None else out | {"q": q}


def _rotated(x, cs, layout, inverse=False):
    """x [tokens, heads, dim] in float32 with its first pairs turned by cs [tokens, pairs, 2]."""
    n = cs.shape[1]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    if inverse:
        s = -s
    turned, rest = x[..., :2 * n], x[..., 2 * n:]
    if layout == "half":
        a, b = turned[..., :n], turned[..., n:]
        return torch.cat((a * c - b * s, b * c + a * s, rest), -1)
    a, b = turned[..., 0::2], turned[..., 1::2]
    return torch.cat((torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2), rest), -1)


def _plain_rope(st, case):
    return _rotated(st["x"].float(), st["table"][st["pos"].long()], case["layout"], case["inverse"]).half()


def _tokens(st):
    """Sequence, number in it and position of each new token."""
    cu, length = st["cu_q"].long(), st["kv_len"].long()
    tok = torch.arange(st["q"].shape[0], device="cuda")
    s = torch.searchsorted(cu[1:], tok, right=True)
    i = tok - cu[s]
    return s, i, length[s] - (cu[s + 1] - cu[s]) + i


def _plain_append(st, case):
    cu, length, slots = st["cu_q"].long(), st["kv_len"].long(), st["slots"].long()
    T, hk, D, fmt = st["k"].shape[0], case["kv_heads"], case["dim"], case["fmt"]
    q, k, v = st["q"], st["k"], st["v"]
    if case["rot"]:
        cs = st["table"][_tokens(st)[2]]
        q = _rotated(q.float(), cs, case["layout"]).half()
        k = _rotated(k.float(), cs, case["layout"]).half()
    before = length - (cu[1:] - cu[:-1])
    # the blocks that the new tokens touch: [sequences, touched]; past the last one it comes again
    touched = (st["max_new"] + 2 * BLOCK - 2) // BLOCK
    blk = torch.minimum((before // BLOCK)[:, None] + torch.arange(touched, device="cuda"), (length - 1)[:, None] // BLOCK)
    p = blk[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")
    old = (p < before[:, None, None])[..., None, None]
    here = (p < length[:, None, None])[..., None, None]
    src = (cu[:-1, None, None] + p - before[:, None, None]).clamp(0, T - 1)
    full = ((blk + 1) * BLOCK <= length[:, None])
    ids = st["block_table"].long().gather(1, blk)
    for name, x in (("k", k), ("v", v)):
        tail = st[name + "_tail"][slots]
        tail = (tail.permute(0, 2, 1, 3) if name == "k" else tail.permute(0, 3, 1, 2))[:, None]
        rows = torch.where(here, torch.where(old, tail, x[src]), torch.zeros((), dtype=x.dtype, device="cuda"))
        f = rows.float()                                    # [sequences, touched, 64, kv heads, dim]
        amax = f.abs().amax((2, 4))
        inv = torch.where(amax > 0, CODE_MAX[fmt] / amax, torch.zeros_like(amax))
        c = f * inv[:, :, None, :, None]
        c = c.round().clamp(-127, 127).to(torch.int8) if fmt == "int8" else c.clamp(-448, 448).to(torch.float8_e4m3fn)
        c = c.view(torch.uint8).permute(*((0, 1, 3, 2, 4) if name == "k" else (0, 1, 3, 4, 2)))
        codes, scale = st[name + "_codes"].view(torch.uint8), st[name + "_scale"]
        codes[ids] = torch.where(full[..., None, None, None], c, codes[ids])
        scale[ids] = torch.where(full[..., None], amax / CODE_MAX[fmt], scale[ids])
        # the tokens of the block that stays open
        p0 = (length // BLOCK * BLOCK)[:, None] + torch.arange(BLOCK, device="cuda")
        stay = ((p0 >= before[:, None]) & (p0 < length[:, None]))[..., None, None]
        src0 = (cu[:-1, None] + p0 - before[:, None]).clamp(0, T - 1)
        now = st[name + "_tail"][slots]
        now = now.permute(0, 2, 1, 3) if name == "k" else now.permute(0, 3, 1, 2)
        now = torch.where(stay, x[src0], now)
        st[name + "_tail"][slots] = now.permute(0, 2, 1, 3) if name == "k" else now.permute(0, 2, 3, 1)
    return _written(st, q if case["rot"] else None)


def _plain_attention(st, case):
    cu, length, slots = st["cu_q"].long(), st["kv_len"].long(), st["slots"].long()
    S, hq, hk, D = case["seqs"], case["heads"], case["kv_heads"], case["dim"]
    g, R = hq // hk, st["max_new"]
    nb = (st["max_len"] + BLOCK - 1) // BLOCK
    ids = st["block_table"][:, :nb].long().clamp(min=0)
    open_ = (torch.arange(nb, device="cuda") == (length // BLOCK)[:, None])[..., None, None, None]
    both = []
    for name in ("k", "v"):
        x = st[name + "_codes"].view(torch.uint8)[ids].view(st[name + "_codes"].dtype).float()
        x = x * st[name + "_scale"][ids][..., None, None]
        x = torch.where(open_, st[name + "_tail"][slots][:, None].float(), x)
        both.append(x.permute(0, 2, 1, 3, 4) if name == "k" else x.permute(0, 2, 1, 4, 3))
    k, v = (x.reshape(S, hk, nb * BLOCK, D) for x in both)
    new = cu[1:] - cu[:-1]
    i = torch.arange(R, device="cuda")
    src = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][src].float().reshape(S, R, hk, g, D).permute(0, 2, 1, 3, 4).reshape(S, hk, R * g, D)
    end = length[:, None] - (new[:, None] - 1 - i if case["causal"] else torch.zeros_like(i))      # [sequences, new]
    see = torch.arange(nb * BLOCK, device="cuda") < end[..., None]
    score = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(D ** -0.5).view(S, hk, R, g, nb * BLOCK)
    score.masked_fill_(~see[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    e = score.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(S, hk, R * g, nb * BLOCK), v).view(S, hk, R, g, D) / total.clamp(min=1e-30)
    s, n, _ = _tokens(st)
    return o.permute(0, 2, 1, 3, 4).reshape(S, R, hq, D)[s, n].half()


EPS = 1e-6


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
    return {"r": r, "h": h.half()}


_own = {"rope": _own_rope, "append": _own_append, "attention": _own_attention, "norm": _own_norm}
_plain = {"rope": _plain_rope, "append": _plain_append, "attention": _plain_attention, "norm": _plain_norm}


# ---------------------------------------------------------------------------------------------------- 64 bits
def _turn64(x, pos, rot, layout, f, mag, sign=1.0):
    """The rotation as a product of complex numbers, in 64 bits."""
    a = pos.double()[:, None] * f.cuda() * sign
    z = torch.polar(torch.full_like(a, mag), a)[:, None, :]
    x, n = x.double(), rot // 2
    y = x.clone()
    if layout == "half":
        w = torch.complex(x[..., :n], x[..., n:rot]) * z
        y[..., :n], y[..., n:rot] = w.real, w.imag
    else:
        w = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * z
        y[..., 0:rot:2], y[..., 1:rot:2] = w.real, w.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        f, mag = _frequencies(case["rot"], case["scaling"], case["factor"])
        return _turn64(st["x"], st["pos"], case["rot"], case["layout"], f, mag, -1.0 if case["inverse"] else 1.0)
    if op == "norm":
        y = st["y"].double()
        if case["post"]:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[1] + EPS) * (st["w_post"].double() + case["offset"])
        if case["gate"] != "none":
            y = y * st["gate"].double()
        r = case["alpha"] * st["r"].double() + case["beta"] * y
        h = r / torch.sqrt((r * r).sum(-1, keepdim=True) / r.shape[1] + EPS) * (st["w_pre"].double() + case["offset"])
        return {"r": r, "h": h}
    new, whole = _lens(case)
    D, hk, fmt = case["dim"], case["kv_heads"], case["fmt"]
    table, slots = st["block_table"].tolist(), st["slots"].tolist()
    if op == "append":
        out = {n: st[n].double() for n in ("k_scale", "v_scale", "k_tail", "v_tail")}
        # codes of eight-bit floats as the values before their rounding; whole codes have no 64-bit value of their own
        for n in ("k_codes", "v_codes"):
            out[n] = st[n].double() if fmt == "e4m3" else None
        f, mag = _frequencies(case["rot"], "none", 1.0) if case["rot"] else (None, 1.0)
        queries, at = [], 0
        for s, (n, w) in enumerate(zip(new, whole)):
            pos = torch.arange(w - n, w, device="cuda")
            k, v = st["k"][at:at + n].double(), st["v"][at:at + n].double()
            if case["rot"]:
                k = _turn64(k, pos, case["rot"], case["layout"], f, mag)
                queries.append(_turn64(st["q"][at:at + n], pos, case["rot"], case["layout"], f, mag))
            at += n
            have = (w - n) % BLOCK              # tokens of the open block that were there
            k = torch.cat((st["k_tail"][slots[s]].double().transpose(0, 1)[:have], k))
            v = torch.cat((st["v_tail"][slots[s]].double().permute(2, 0, 1)[:have], v))
            first = (w - n) // BLOCK
            for j in range(k.shape[0] // BLOCK):
                b = table[s][first + j]
                for x, name in ((k, "k"), (v, "v")):
                    t = x[j * BLOCK:(j + 1) * BLOCK]
                    sc = t.abs().amax((0, 2)) / CODE_MAX[fmt]
                    out[name + "_scale"][b] = sc
                    if fmt == "e4m3":
                        c = t / torch.where(sc > 0, sc, torch.ones_like(sc))[None, :, None]
                        out[name + "_codes"][b] = c.transpose(0, 1) if name == "k" else c.permute(1, 2, 0)
            done = k.shape[0] // BLOCK * BLOCK
            keep = have if not done else 0
            for t in range(done + keep, k.shape[0]):
                out["k_tail"][slots[s]][:, t - done] = k[t]
                out["v_tail"][slots[s]][:, :, t - done] = v[t]
        return out | ({"q": torch.cat(queries)} if case["rot"] else {})
    parts, at, g = [], 0, case["heads"] // hk
    for s, (n, w) in enumerate(zip(new, whole)):
        full = w // BLOCK
        ids = torch.tensor(table[s][:full], dtype=torch.long, device="cuda")
        head = []
        for h in range(hk):
            k = st["k_codes"].view(torch.uint8)[ids, h].view(st["k_codes"].dtype).double() * st["k_scale"][ids, h].double()[:, None, None]
            v = st["v_codes"].view(torch.uint8)[ids, h].view(st["v_codes"].dtype).double() * st["v_scale"][ids, h].double()[:, None, None]
            k = torch.cat((k.reshape(-1, D), st["k_tail"][slots[s], h].double()[:w - full * BLOCK]))
            v = torch.cat((v.transpose(1, 2).reshape(-1, D), st["v_tail"][slots[s], h].double().t()[:w - full * BLOCK]))
            q = st["q"][at:at + n, h * g:(h + 1) * g].double()
            t = q.reshape(n * g, D) @ k.t() / math.sqrt(D)
            if case["causal"]:
                last = (w - n + torch.arange(n, device="cuda"))[:, None].expand(n, g).reshape(-1)
                t.masked_fill_(torch.arange(w, device="cuda") > last[:, None], -math.inf)
            head.append((torch.softmax(t, -1) @ v).view(n, g, D))
        parts.append(torch.cat(head, 1))
        at += n
    return torch.cat(parts)
