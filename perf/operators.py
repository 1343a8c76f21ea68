"""The token-stream operators, measured: rotary positions of token tensors, the
append to a paged KV cache, and attention over that cache.

Where `own` is true, run() calls this repository's package; where it is false
it computes the same in elementary torch operations (fp32, angles in fp64).
Every case is one call on a ragged batch of sequences whose keys and values
live in pages of a shared pool. Lengths are a fixed function of the case;
values, and which pages a sequence owns, come from the seed.
"""
import math
import random

import numpy as np
import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rope(kind="none", rot=0, scale=1.0, original=0, amplitude=1.0, theta=10000.0):
    return {"rope": kind, "rot": rot, "rope_scale": scale, "rope_original": original, "amplitude": amplitude,
            "theta": theta}


def _attention(name, *, B, q, kv, Hq, Hkv, D, dtype, page, window=0, sink=0, cap=0.0, bias=False, prefix=0, **rope):
    return {"name": name, "op": "attention", "B": B, "q": q, "kv": kv, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype,
            "page": page, "window": window, "sink": sink, "cap": cap, "bias": bias, "prefix": prefix,
            **_rope(**rope)}


def _append(name, *, B, q, kv, Hkv, D, dtype, page, **rope):
    return {"name": name, "op": "append", "B": B, "q": q, "kv": kv, "Hkv": Hkv, "D": D, "dtype": dtype, "page": page,
            **_rope(**rope)}


def _rotary(name, *, T, H, D, dtype, far, transpose, **rope):
    return {"name": name, "op": "rope", "T": T, "H": H, "D": D, "dtype": dtype, "far": far, "transpose": transpose,
            **_rope(**rope)}


def listed():
    return [
        # one user's stream, one new token, a short history: latency
        _attention("decode-one-bf16", B=1, q=1, kv=700, Hq=32, Hkv=8, D=128, dtype="bf16", page=16,
                   kind="half", rot=128),
        # a served batch at ordinary lengths over the 8-bit cache
        _attention("decode-batch-e4m3", B=48, q=1, kv=8000, Hq=32, Hkv=8, D=128, dtype="e4m3", page=16,
                   kind="half", rot=128),
        # few streams with very long histories, many query heads to a key head
        _attention("decode-long-e4m3", B=4, q=1, kv=131000, Hq=64, Hkv=8, D=128, dtype="e4m3", page=64,
                   kind="interleaved", rot=128, scale=0.25, original=32768, amplitude=1.1386),
        # three tokens at a time (drafted tokens under check), sinks and a window, capped scores, one key head each
        _attention("decode-window-bf16", B=9, q=3, kv=5001, Hq=12, Hkv=12, D=64, dtype="bf16", page=32,
                   window=4097, sink=5, cap=30.0),
        # prompts of several users computed at once, part of each in the cache already
        _attention("prefill-bf16", B=3, q=2311, kv=4333, Hq=32, Hkv=8, D=128, dtype="bf16", page=16,
                   kind="half", rot=128),
        # one chunk of a long prompt over the 8-bit cache
        _attention("chunk-e4m3", B=1, q=1024, kv=32768, Hq=32, Hkv=8, D=128, dtype="e4m3", page=64),
        # a prefix that every token sees, and a bias that grows with the distance
        _attention("prefix-bias-bf16", B=5, q=777, kv=1500, Hq=12, Hkv=12, D=64, dtype="bf16", page=16,
                   bias=True, prefix=257),
        # the append of one token of every sequence of a served batch
        _append("append-batch-e4m3", B=48, q=1, kv=8000, Hkv=8, D=128, dtype="e4m3", page=16, kind="half", rot=128),
        # the append of whole prompts
        _append("append-prompts-e4m3", B=7, q=4096, kv=6001, Hkv=8, D=128, dtype="e4m3", page=64,
                kind="half", rot=128),
        _append("append-prompts-bf16", B=5, q=1560, kv=3333, Hkv=12, D=128, dtype="bf16", page=16,
                kind="interleaved", rot=96),
        # the queries of one step
        _rotary("rope-step", T=48, H=32, D=128, dtype="bf16", far=8000, transpose=False, kind="half", rot=128),
        # gradients of a long training batch, half of each head rotated
        _rotary("rope-grad-long", T=32768, H=12, D=128, dtype="f32", far=1000000, transpose=True,
                kind="interleaved", rot=64, scale=0.125),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rope(rng, D):
    kind = rng.choice(["half", "interleaved"])
    rot = rng.choice([r for r in (32, 48, 64, 96, 128) if r <= D])
    if rng.random() < 0.3:
        return dict(kind=kind, rot=rot, scale=rng.choice([0.125, 0.25, 0.5]), original=rng.choice([0, 4096, 32768]),
                    amplitude=rng.choice([1.0, 1.1386]))
    return dict(kind=kind, rot=rot, theta=rng.choice([10000.0, 500000.0]))


def draw(rng: random.Random):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "append", "append", "rope"])
    D = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    if Hkv * group > 64:
        group = 4
    if op == "rope":
        c = _rotary("", T=_spread(rng, 1, 30000), H=rng.choice([1, 5, 8, 12]), D=D, dtype=rng.choice(["bf16", "f32"]),
                    far=_spread(rng, 100, 1000000), transpose=rng.random() < 0.5, **_draw_rope(rng, D))
    elif op == "append":
        B = _spread(rng, 1, 64)
        q = _spread(rng, 1, max(1, 16000 // B))
        c = _append("", B=B, q=q, kv=q + _spread(rng, 1, 4000), Hkv=Hkv, D=D, dtype=dtype, page=page,
                    **_draw_rope(rng, D))
    else:
        mods = {}
        if op == "decode":
            B = _spread(rng, 1, 64)
            q = rng.choice([1, 1, 1, 2, 5])
            kv = _spread(rng, 33, min(100000, 300000 // B))
        else:
            B = _spread(rng, 1, 6)
            q = _spread(rng, 17, 2000 // B)
            kv = q + _spread(rng, 1, 5000 // B)
        if rng.random() < 0.4:
            mods["window"] = _spread(rng, 16, kv)
            mods["sink"] = rng.choice([0, 3, 64])
        if rng.random() < 0.3:
            mods["cap"] = rng.choice([20.0, 50.0])
        if rng.random() < 0.3:
            mods["bias"] = True
        if rng.random() < 0.3:
            mods["prefix"] = _spread(rng, 1, kv)
        if rng.random() < 0.6:
            mods.update(_draw_rope(rng, D))
        c = _attention("", B=B, q=q, kv=kv, Hq=Hkv * group, Hkv=Hkv, D=D, dtype=dtype, page=page, **mods)
    del c["name"]
    return c


def _lengths(case):
    """(new tokens, length with them) of every sequence: the first sequence has the case's largest of both."""
    r = random.Random(1234567 + case["B"] * 7919 + case["q"] * 104729 + case["kv"])
    q, kv = [case["q"]], [case["kv"]]
    for b in range(1, case["B"]):
        n = case["q"] if case["q"] <= 8 else r.randint(1, case["q"])
        q.append(n)
        kv.append(r.randint(min(case["kv"], max(n, case["kv"] // 4)), case["kv"]))
        if b == 5:  # a slot of the batch that holds no sequence at present
            q[b], kv[b] = 0, 0
    return q, kv


def _prefixes(case):
    return [min(case["prefix"], n) for n in _lengths(case)[1]]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _two_power(amax):
    """The smallest power of two s with 448 s >= amax (0 for 0)."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126))
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _fill(shape, dtype, g, spread):
    """Pages of finite values: (values or codes, scales or None). [n_pages][H][page][D]"""
    n, H, page, D = shape
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp2(spread * torch.randn((1, H, 1, D), generator=g, device="cuda"))
    if dtype == "bf16":
        return x.bfloat16(), None
    s = _two_power(x.abs().amax(dim=(2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    D = case["D"]
    s = {"case": case}
    if case["op"] == "rope":
        t = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["x"] = torch.randn((case["T"], case["H"], D), generator=g, device="cuda").to(t)
        s["pos"] = torch.randint(0, case["far"], (case["T"],), generator=g, device="cuda", dtype=torch.int32)
        if own:
            s["rope"] = _own_rope(case)
        return s
    B, page, Hkv = case["B"], case["page"], case["Hkv"]
    q, kv = _lengths(case)
    pages = [-(-n // page) for n in kv]
    total, rows = sum(pages) + 3, sum(q)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
    s["table"] = table
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor(np.cumsum([0] + q), dtype=torch.int32, device="cuda")
    s["k"], s["k_scale"] = _fill((total, Hkv, page, D), case["dtype"], g, 0.5)
    s["v"], s["v_scale"] = _fill((total, Hkv, page, D), case["dtype"], g, 0.2)
    if case["op"] == "append":
        s["k_new"] = (1.3 * torch.randn((rows, Hkv, D), generator=g, device="cuda")).bfloat16()
        s["v_new"] = torch.randn((rows, Hkv, D), generator=g, device="cuda").bfloat16()
    else:
        s["q"] = (1.5 * torch.randn((rows, case["Hq"], D), generator=g, device="cuda")).bfloat16()
        s["prefix"] = torch.tensor(_prefixes(case), dtype=torch.int32, device="cuda") if case["prefix"] else None
        s["slopes"] = _slopes(case) if case["bias"] else None
    if own:  # the handles that a serving loop keeps
        import sink_window_attention_b200 as swa
        s["cache"] = swa.PagedKVCache(total, page, Hkv, D, "fp8" if case["dtype"] == "e4m3" else "bf16")
        for name in ("k", "v", "k_scale", "v_scale"):
            if s[name] is not None:
                getattr(s["cache"], name).copy_(s[name])
        s["batch"] = swa.TokenBatch(s["q_start"], s["kv_len"], s["table"], max_q=max(q), max_kv=max(kv))
        s["rope"] = _own_rope(case)
        if case["op"] == "attention":
            s["scores"] = swa.Scores(window=case["window"], n_sink=case["sink"], prefix_len=s["prefix"],
                                     soft_cap=case["cap"], slopes=s["slopes"])
    return s


def _own_rope(case):
    import sink_window_attention_b200 as swa
    if case["rope"] == "none":
        return None
    return swa.TokenRope(case["rot"], theta0=case["theta"], layout=case["rope"], scale=case["rope_scale"],
                         original_len=case["rope_original"], amplitude=case["amplitude"])


def _slopes(case):
    """One slope per query head, a geometric series."""
    return [2.0 ** (-8.0 * (h + 1) / case["Hq"]) for h in range(case["Hq"])]


# ---------------------------------------------------------------------------
# run
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import sink_window_attention_b200 as swa
    case = s["case"]
    if case["op"] == "rope":
        return swa.token_rope_apply(s["x"], s["pos"], s["rope"], transpose=case["transpose"])
    if case["op"] == "append":
        c = s["cache"]
        swa.paged_append(c, s["batch"], s["k_new"], s["v_new"], s["rope"])
        return _whole(case, c.k, c.v, c.k_scale, c.v_scale)
    return swa.paged_attention(s["q"], s["cache"], s["batch"], s["rope"], s["scores"])


def _whole(case, k, v, ks, vs):
    if case["dtype"] == "bf16":
        return [k, v]
    return [k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs]


def _angle_table(case, pos):
    """cos and sin, fp32 [tokens][rot / 2], of angles taken in fp64."""
    half = case["rot"] // 2
    i = torch.arange(half, dtype=torch.float64, device=pos.device)
    w = torch.exp2(-(2.0 * i / case["rot"]) * math.log2(case["theta"]))
    keep = torch.zeros_like(w)
    if case["rope_original"]:
        turns = case["rope_original"] * w / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    w = w * (keep + (1.0 - keep) * case["rope_scale"])
    a = pos.double()[:, None] * w
    return (torch.cos(a) * case["amplitude"]).float(), (torch.sin(a) * case["amplitude"]).float()


def _rotate(case, x, pos, transpose=False):
    """x fp32 [tokens][heads][D], rotated at its tokens' positions."""
    if case["rope"] == "none":
        return x
    c, sn = _angle_table(case, pos)
    c, sn = c[:, None, :], (-sn if transpose else sn)[:, None, :]
    rot, half = case["rot"], case["rot"] // 2
    head, tail = x[..., :rot], x[..., rot:]
    if case["rope"] == "half":
        a, b = head[..., :half], head[..., half:]
        y = torch.cat([a * c - b * sn, a * sn + b * c], dim=-1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * c - b * sn, a * sn + b * c], dim=-1).flatten(-2)
    return torch.cat([y, tail], dim=-1)


def _token_places(s):
    """(sequence, position) of every new token."""
    start, kv = s["q_start"].long(), s["kv_len"].long()
    n = start[1:] - start[:-1]
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=n.device), n, output_size=sum(_lengths(s["case"])[0]))
    pos = kv[seq] - n[seq] + (torch.arange(seq.numel(), device=n.device) - start[:-1][seq])
    return seq, pos


def _run_plain(s):
    case = s["case"]
    if case["op"] == "rope":
        x = s["x"]
        return _rotate(case, x.float(), s["pos"], case["transpose"]).to(x.dtype)
    if case["op"] == "append":
        return _plain_append(s)
    return _plain_attention(s)


def _plain_append(s):
    case = s["case"]
    seq, pos = _token_places(s)
    page = case["page"]
    to, slot = s["table"][seq, pos // page].long(), pos % page
    k, v = _rotate(case, s["k_new"].float(), pos), s["v_new"].float()
    if case["dtype"] == "bf16":
        s["k"][to, :, slot] = k.bfloat16()
        s["v"][to, :, slot] = v.bfloat16()
        return _whole(case, s["k"], s["v"], None, None)
    # the touched pages, one after the other; `touched`: their numbers
    flag = torch.zeros(s["k"].shape[0], dtype=torch.bool, device=to.device)
    flag[to] = True
    touched = flag.nonzero()[:, 0]
    where = torch.zeros_like(flag, dtype=torch.int64)
    where[touched] = torch.arange(touched.numel(), device=to.device)
    new = torch.zeros((touched.numel(), page), dtype=torch.bool, device=to.device)
    new[where[to], slot] = True
    first = torch.where(new.any(1), new.to(torch.int8).argmax(1), page)  # first new slot: those before it hold older tokens
    old = torch.arange(page, device=to.device)[None, :] < first[:, None]
    for codes, scales, x in ((s["k"], s["k_scale"], k), (s["v"], s["v_scale"], v)):
        block = torch.zeros((touched.numel(), case["Hkv"], page, case["D"]), device=to.device)
        block[where[to], :, slot] = x
        before = torch.where(first[:, None] > 0, scales[touched], torch.zeros((), device=to.device))
        scale = torch.maximum(before, _two_power(block.abs().amax(dim=(2, 3))))
        inverse = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))[:, :, None, None]
        was = codes[touched].view(torch.float8_e4m3fn).float()
        again = (was * (before[:, :, None, None] * inverse)).to(torch.float8_e4m3fn)
        fresh = (block * inverse).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        got = torch.where(old[:, None, :, None], again.view(torch.uint8), codes[touched])
        codes[touched] = torch.where(new[:, None, :, None], fresh.view(torch.uint8), got)
        scales[touched] = scale
    return _whole(case, s["k"], s["v"], s["k_scale"], s["v_scale"])


def _pages_of(case, pool, scales, table):
    """fp32 [B][Hkv][tokens][D] of the pages of every sequence."""
    at = table.long().clamp(min=0)
    x = pool[at]
    if case["dtype"] == "e4m3":
        x = x.view(torch.float8_e4m3fn).float() * scales[at][..., None, None]
    return x.float().transpose(1, 2).flatten(2, 3)


def _plain_attention(s):
    case = s["case"]
    B, Q, Hq, Hkv, D = case["B"], case["q"], case["Hq"], case["Hkv"], case["D"]
    seq, pos = _token_places(s)
    within = torch.arange(seq.numel(), device=seq.device) - s["q_start"].long()[seq]
    q = _rotate(case, s["q"].float(), pos)
    rows = torch.zeros((B, Q, Hq, D), device=q.device)
    rows[seq, within] = q
    at = torch.full((B, Q), -1, dtype=torch.int64, device=q.device)
    at[seq, within] = pos
    k = _pages_of(case, s["k"], s["k_scale"], s["table"])
    v = _pages_of(case, s["v"], s["v_scale"], s["table"])
    rows = rows.reshape(B, Q, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    scores = (rows @ k.transpose(-1, -2)) * D ** -0.5
    scores = scores.view(B, Hkv, Hq // Hkv, Q, -1)
    if case["cap"]:
        scores = torch.tanh_(scores / case["cap"]) * case["cap"]
    j = torch.arange(scores.shape[-1], device=q.device)
    p = at[:, :, None]
    if case["bias"]:
        slopes = torch.tensor(s["slopes"], device=q.device).view(1, Hkv, -1, 1, 1)
        scores = scores - slopes * (p - j).abs().float()[:, None, None]
    seen = j <= p
    if case["window"]:
        seen = seen & ((j > p - case["window"]) | (j < case["sink"]))
    if case["prefix"]:
        seen = seen | (j < s["prefix"][:, None, None])
    seen = (seen & (j < s["kv_len"][:, None, None]))[:, None, None]
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(scores - top)
    weights = e / e.sum(-1, keepdim=True).clamp(min=1e-37)
    out = (weights.view(B, Hkv, -1, weights.shape[-1]) @ v).view(B, Hkv, Hq // Hkv, Q, D)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D)
    return out[seq, within].bfloat16()


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    D = case["D"]
    if case["op"] == "rope":
        n = case["T"] * case["H"] * D
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4) + 4 * case["T"], "flops": 3 * n}
    q, kv = _lengths(case)
    size = 1 if case["dtype"] == "e4m3" else 2
    if case["op"] == "append":
        n = sum(q) * case["Hkv"] * D * 2
        pages = sum((-(-l // case["page"]) - (l - m) // case["page"]) if m else 0 for m, l in zip(q, kv))
        return {"bytes": n * (2 + size) + (pages * case["Hkv"] * 8 if size == 1 else 0), "flops": 4 * n}
    pairs, keys = 0, 0
    for m, l, pre in zip(q, kv, _prefixes(case)):
        if not m:
            continue
        p = np.arange(l - m, l, dtype=np.int64)
        low = np.maximum(0, p - case["window"] + 1) if case["window"] else np.zeros_like(p)
        always = np.maximum(pre, np.minimum(case["sink"] if case["window"] else 0, p + 1))  # keys [0, always) are seen
        pairs += int((always + np.maximum(0, p + 1 - np.maximum(low, always))).sum())
        keys += int(always[-1] + max(0, l - max(int(low[0]), int(always[-1]))))
    scales = keys / case["page"] * case["Hkv"] * 8 if size == 1 else 0
    return {"bytes": keys * case["Hkv"] * D * 2 * size + scales + sum(q) * case["Hq"] * D * 4,
            "flops": 4.0 * pairs * case["Hq"] * D}


# ---------------------------------------------------------------------------
# the definition, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turn(case, s["x"].double(), s["pos"].double(), -1.0 if case["transpose"] else 1.0)
    if case["op"] == "append":
        return _exact_append(case, s)
    return _exact_attention(case, s)


def _exact_turn(case, x, pos, sign=1.0):
    """Each pair (a, b) of a head as the complex number a + ib, times amplitude * exp(i sign angle)."""
    if case["rope"] == "none":
        return x
    y = x.clone()
    for n in range(case["rot"] // 2):
        w = case["theta"] ** (-2.0 * n / case["rot"])
        keep = 0.0
        if case["rope_original"]:
            keep = min(1.0, max(0.0, (case["rope_original"] * w / (2.0 * math.pi) - 1.0) / 31.0))
        w *= keep + (1.0 - keep) * case["rope_scale"]
        a, b = (2 * n, 2 * n + 1) if case["rope"] == "interleaved" else (n, n + case["rot"] // 2)
        z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.full_like(pos, case["amplitude"]), sign * w * pos)[:, None]
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_e4m3(x):
    """The nearest E4M3 value (ties to even, at most 448)."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(case, s):
    q, kv = _lengths(case)
    page, start = case["page"], 0
    small = case["dtype"] == "e4m3"
    out = []
    for name in ("k", "v"):
        pool = (s[name].view(torch.float8_e4m3fn) if small else s[name]).double()
        out.append([pool, s[name + "_scale"].double() if small else None])
    for b, (m, l) in enumerate(zip(q, kv)):
        pos = torch.arange(l - m, l, device="cuda", dtype=torch.float64)
        rows = slice(start, start + m)
        fresh = (_exact_turn(case, s["k_new"][rows].double(), pos), s["v_new"][rows].double())
        start += m
        table = s["table"][b].tolist()
        t = l - m
        while t < l:  # one page after the other
            off, n = t % page, min(page - t % page, l - t)
            to = table[t // page]
            for (pool, scales), x in zip(out, fresh):
                x = x[t - (l - m):t - (l - m) + n].transpose(0, 1)  # [Hkv][n][D]
                if small:
                    need = x.abs().amax(dim=(1, 2))
                    two = torch.exp2(torch.ceil(torch.log2((need / 448).clamp(min=2.0 ** -126))))
                    two = torch.where(need > 0, two, torch.zeros_like(two))
                    was = scales[to] if off else torch.zeros_like(two)
                    scale = torch.maximum(was, two)
                    safe = torch.where(scale > 0, scale, torch.ones_like(scale))[:, None, None]
                    pool[to, :, :off] = _exact_e4m3(pool[to, :, :off] * was[:, None, None] / safe)
                    x = _exact_e4m3(x / safe)
                    scales[to] = scale
                pool[to, :, off:off + n] = x
            t += n
    if small:
        return [out[0][0], out[1][0], out[0][1], out[1][1]]
    return [out[0][0], out[1][0]]


def _exact_attention(case, s):
    q, kv = _lengths(case)
    D, group, start = case["D"], case["Hq"] // case["Hkv"], 0
    if sum(m * l for m, l in zip(q, kv)) * case["Hq"] * D > 3e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, (m, l) in enumerate(zip(q, kv)):
        if not m:
            continue
        rows = slice(start, start + m)
        start += m
        p = torch.arange(l - m, l, device="cuda")
        j = torch.arange(l, device="cuda")
        mask = j[None, :] <= p[:, None]
        if case["window"]:
            mask &= (p[:, None] - j[None, :] < case["window"]) | (j[None, :] < case["sink"])
        if case["prefix"]:
            mask |= j[None, :] < _prefixes(case)[b]
        query = _exact_turn(case, s["q"][rows].double(), p.double())
        pages = s["table"][b, :-(-l // case["page"])].long()
        for h in range(case["Hkv"]):
            kvs = []
            for name in ("k", "v"):
                x = s[name][pages, h]
                if case["dtype"] == "e4m3":
                    x = x.view(torch.float8_e4m3fn).double() * s[name + "_scale"][pages, h].double()[:, None, None]
                kvs.append(x.double().reshape(-1, D)[:l])
            for g in range(h * group, (h + 1) * group):
                z = query[:, g] @ kvs[0].T / math.sqrt(D)
                if case["cap"]:
                    z = case["cap"] * torch.tanh(z / case["cap"])
                if case["bias"]:
                    z = z - s["slopes"][g] * (p[:, None] - j[None, :]).abs()
                out[rows, g] = torch.softmax(z.masked_fill(~mask, -math.inf), dim=-1) @ kvs[1]
    return out
