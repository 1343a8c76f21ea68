"""Attention over a paged pool where its roundings, ranges and masks can go wrong,
as a whole (tests/paged_checks.py) and against the fp64 oracle."""
import numpy as np
import pytest
import torch

import sink_window_attention_b200 as swa
from oracle import tokens
from tests.paged_checks import norm_error, norm_limit
from tests.test_gpu_tokens import MODS, SHAPES, Setup, f64, i32

pytestmark = pytest.mark.gpu


def expected(s, q, rope=None, **kw):
    """The oracle's rows (and lse, and what bounds need) of a whole call."""
    parts, at = [], 0
    for b, n in enumerate(s.news):
        x = f64(q[at:at + n])
        if rope is not None:
            x = tokens.rotate(x, np.arange(s.lens[b] - n, s.lens[b]), tokens.frequencies(rope.rot_dim), rope.layout)
        (k, there), (v, _) = s.keys(b, "k"), s.keys(b, "v")
        args = {**kw, "prefix": kw["prefix"][b]} if "prefix" in kw else kw
        parts.append(tokens.attend(x, k, v, s.lens[b], exists=there, **args))
        at += n
    return [np.concatenate(p) for p in zip(*parts)]


# ---------------------------------------------------------------------------
# one key with nearly all of the mass
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("gap", [11.0, 13.5, 15.4])
@pytest.mark.parametrize("sink", [0, 1390])
def test_tail_behind_one_key(dtype, D, new, gap, sink):
    """A pinned token with nearly all of the mass and a value of zero: the output is the
    tail of some 1400 equal weights e^-gap below it. Each is rounded to bf16 (2^-8) or to
    fp16: 2^-11, or half a step of the subnormals, 2^-31 of the largest weight. All are
    equal, so their errors add up. The pinned key comes first, or last (the tail is then
    made of fp16 normals, which shrink in fp32). So many units that no range is split:
    the sink and its tail meet in one sum."""
    B, H, n = (3 if new == 1 else 1), 128, 1400 + new
    s = Setup([n] * B, [n] * B, H, D, dtype, 64)
    k = torch.zeros((B, n, H, D), device="cuda")
    v = 1 + torch.randn((B, n, H, D), generator=torch.Generator(device="cuda").manual_seed(D), device="cuda")
    k[:, sink] = 8.0
    v[:, sink] = 0.0
    swa.paged_append(s.cache, s.batch(), k.view(-1, H, D).bfloat16(), v.view(-1, H, D).bfloat16())
    s.take()
    s.news = [new] * B
    q = torch.ones((B * new, H, D), device="cuda").bfloat16()
    lse = torch.empty((B * new, H), device="cuda")
    got = f64(swa.paged_attention(q, s.cache, s.batch(), None, swa.Scores(softmax_scale=gap / (8.0 * D)), lse=lse))
    want, total = np.zeros((B, new, H, D)), np.zeros((B, new, H))
    w = np.full(n, np.exp(-gap))
    w[sink] = 1.0
    for b in range(B):
        vals = s.keys(b, "v")[0].reshape(n, H * D)
        for i in range(new):
            seen = n - new + i + 1
            total[b, i] = w[:seen].sum()
            want[b, i] = (w[:seen] @ vals[:seen] / w[:seen].sum()).reshape(H, D)
    want = want.reshape(got.shape)
    rel = 2.0**-8 if dtype == "bf16" else max(2.0**-11, 2.0**-31 * np.exp(gap))
    # and the output's rounding; the scale is held in fp32 (a score of gap is off by 2^-23 gap, ex2 by 2^-22)
    assert norm_error(got, want) <= rel + 1.35 * 1.7e-3 + 4e-5
    assert np.abs(f64(lse) - gap - np.log(total.reshape(lse.shape))).max() <= 4e-5


# ---------------------------------------------------------------------------
# scales
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("new", [1, 60, 140])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mods", [dict(window=40, n_sink=3), dict(window=1100), dict(window=1100, n_sink=3),
                                  dict(window=1033, n_sink=17, cap=4.0)])
def test_scales_of_keys_that_no_row_sees(new, page, D, mods):
    """Mapped pages before the window, or between the sinks and it, with NaN or
    infinite scales (pages given back): what their places hold does not matter."""
    s = Setup([1900, 1510], [new, new], 2, D, "fp8", page)
    s.fill(3)
    for b, n in enumerate(s.lens):
        lo = n - new - mods["window"] + 1  # the first key that the window of the first row reaches
        for pg in range(-(-mods.get("n_sink", 0) // page), lo // page):
            at = int(s.table[b, pg])
            for name in ("k_scale", "v_scale"):
                getattr(s.cache, name)[at] = float("nan") if pg % 2 else float("inf")
            s.cache.k[at] = 0x7F
            s.cache.v[at] = 0x7F
    q = torch.randn((2 * new, 4, D), device="cuda").bfloat16()
    out = f64(swa.paged_attention(q, s.cache, s.batch(), None, swa.Scores(**{("soft_cap" if a == "cap" else a): x for a, x in mods.items()})))
    for x in (s.pool.ks, s.pool.vs, s.pool.k, s.pool.v):
        x[~np.isfinite(x)] = 0.0
    want = expected(s, q, **mods)[0]
    assert norm_error(out, want) <= norm_limit("fp8", 8 * new)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 60, 140])
@pytest.mark.parametrize("power", [-100, -70, 75, 110])
def test_values_far_from_one(D, new, power):
    """V of 2^-100 to 2^110 in every page: scales beyond what a fp16 product holds."""
    s = Setup([300, 70], [300, 70], 2, D, "fp8", 32)
    g = torch.Generator(device="cuda").manual_seed(power + 200)
    k = torch.randn((370, 2, D), generator=g, device="cuda").bfloat16()
    v = (torch.randn((370, 2, D), generator=g, device="cuda") * 2.0**power).bfloat16()
    swa.paged_append(s.cache, s.batch(), k, v)
    s.take()
    s.news = [min(new, 300), min(new, 70)]
    q = torch.randn((sum(s.news), 4, D), generator=g, device="cuda").bfloat16()
    out = f64(swa.paged_attention(q, s.cache, s.batch()))
    want = expected(s, q)[0]
    assert norm_error(out * 2.0**-power, want * 2.0**-power) <= norm_limit("fp8", out.shape[0] * 4)


# ---------------------------------------------------------------------------
# caps
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 140])
@pytest.mark.parametrize("cap", [0.5, 30.0, 300.0, 1e4, 1e6, 1e30])
def test_caps_far_above_the_scores(dtype, D, new, cap):
    """cap * tanh(x / cap) keeps x's relative precision where the cap is far above it:
    lse within 1e-5 (1 + |x|) of the definition's, whatever the cap."""
    s = Setup([500], [500], 2, D, dtype, 32)
    s.fill(7)
    s.news = [new]
    q = torch.randn((new, 4, D), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    lse = torch.empty((new, 4), device="cuda")
    out = f64(swa.paged_attention(q, s.cache, s.batch(), None, swa.Scores(soft_cap=cap), lse=lse))
    want, ref, _, _ = expected(s, q, cap=cap)
    assert np.abs(f64(lse) - ref).max() <= 3e-5 * (1 + np.abs(ref).max())
    assert norm_error(out, want) <= norm_limit(dtype, 4 * new)


# ---------------------------------------------------------------------------
# outputs as a whole
# ---------------------------------------------------------------------------
LONG = [  # few rows: pieces joined in a cluster, and through the workspace
    ([1500], [1], 2, 4, 64, 16),
    ([2000, 1800, 40], [2, 1, 1], 4, 2, 128, 64),
    ([20011], [1], 2, 8, 128, 64),
    ([9000, 33000], [1, 3], 1, 5, 64, 128),
]


def growing(s, seed):
    """Keys whose size grows along a sequence, so that pieces of it weigh differently;
    values of mean zero."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(s.lens)
    at = torch.cat([torch.linspace(0.4, 1.2, m) for m in s.lens]).cuda()[:, None, None]
    k = (torch.randn((n, s.H, s.D), generator=g, device="cuda") * at).bfloat16()
    v = torch.randn((n, s.H, s.D), generator=g, device="cuda").bfloat16()
    swa.paged_append(s.cache, s.batch(news=s.lens), k, v)
    s.take()


@pytest.mark.parametrize("lens,news,H,group,D,page", SHAPES + LONG)
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("mod", list(MODS))
def test_norm_of_the_error(lens, news, H, group, D, page, dtype, mod):
    s = Setup(lens, news, H, D, dtype, page, seed=3, garbage=True)
    growing(s, 17)
    kw = dict(MODS[mod])
    Hq = H * group
    if kw.pop("bias", False):
        kw["slopes"] = [float(2.0 ** (-1 - h)) for h in range(Hq)]
    if kw.pop("prefix", False):
        kw["prefix"] = [n // 2 + 1 if b % 2 == 0 else 0 for b, n in enumerate(lens)]
    rope = swa.TokenRope(64) if mod == "plain" else swa.TokenRope(32, layout="interleaved") if mod == "sink" else None
    g = torch.Generator(device="cuda").manual_seed(23)
    q = torch.randn((sum(news), Hq, D), generator=g, device="cuda").bfloat16()
    sc = swa.Scores(softmax_scale=kw.get("scale", 0.0), window=kw.get("window", 0), n_sink=kw.get("n_sink", 0),
                    soft_cap=kw.get("cap", 0.0), slopes=kw.get("slopes"),
                    prefix_len=i32(kw["prefix"]) if "prefix" in kw else None)
    out = f64(swa.paged_attention(q, s.cache, s.batch(), rope, sc))
    want = expected(s, q, rope, **kw)[0]
    one_term = rope is not None and max(news) * group > 8
    assert norm_error(out, want) <= norm_limit(dtype, sum(news) * Hq, 1.2 if one_term else 0.0)
    assert swa.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 140])
def test_norm_of_the_error_where_pages_are_powers_of_two_apart(dtype, D, new):
    """Values 2^-20 to 2^20 by page, and keys that grow: each row's output is that of the
    few pages that count for it."""
    s = Setup([1700], [1700], 2, D, dtype, 16, garbage=True)
    g = torch.Generator(device="cuda").manual_seed(6)
    k = torch.randn((1700, 2, D), generator=g, device="cuda") * torch.linspace(0.1, 2, 1700, device="cuda")[:, None, None]
    v = torch.randn((1700, 2, D), generator=g, device="cuda")
    v = v * torch.exp2(((torch.arange(1700, device="cuda") // 16) * 7 % 41 - 20).float())[:, None, None]
    swa.paged_append(s.cache, s.batch(), k.bfloat16(), v.bfloat16())
    s.take()
    s.news = [new]
    q = torch.randn((new, 4, D), generator=g, device="cuda").bfloat16()
    out = f64(swa.paged_attention(q, s.cache, s.batch()))
    assert norm_error(out, expected(s, q)[0]) <= norm_limit(dtype, 4 * new)


@pytest.mark.parametrize("rot,layout", [(64, "half"), (32, "interleaved"), (16, "half")])
@pytest.mark.parametrize("H,group,new", [(2, 4, 140), (1, 1, 300)])
def test_rotated_queries_of_large_scores(rot, layout, H, group, new):
    """Heads of 64 over a bf16 pool, scores of standard deviation 3: a rotated q in one
    bf16 term is off by 3.3 R of the output, in two by 1.4 R, whichever kernel is taken."""
    s = Setup([1500 + new], [1500 + new], H, 64, "bf16", 16, garbage=True)
    s.fill(9)
    s.news = [new]
    rope = swa.TokenRope(rot, layout=layout)
    q = 3 * torch.randn((new, H * group, 64), generator=torch.Generator(device="cuda").manual_seed(8), device="cuda")
    q = q.bfloat16()
    out = f64(swa.paged_attention(q, s.cache, s.batch(), rope))
    assert norm_error(out, expected(s, q, rope)[0]) <= norm_limit("bf16", new * H * group)
