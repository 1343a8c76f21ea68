"""Token streams on the GPU against the fp64 oracle: rotary positions, the append
to a paged pool, attention over it, and a run of the three together.

Tolerances. One rounding to a type is off by at most half a step: bf16 2^-8, fp16
2^-11, fp32 2^-24 of the value. fp32 rotations: the angle is within 2^-25 of a
turn's 2 pi and the sine and cosine within a few 2^-24, so a rotated element is
within 1e-6 * amplitude * (|a| + |b|) of its pair.
Attention, elementwise: out = sum p v / sum p. Rounding q's elements moves a score
by at most eps = u_q * sum_d |q_d k_d| * scale (+ 2^-20 of that for fp32 sums and the
cap's tanh, 1e-5 more with a cap), hence every weight by a factor within e^+-2eps;
rounding the weights moves them by u_p; so |error| <= (e^2eps - 1 + u_p + 1e-5) *
sum_j p_j |v_j| + 2^-8 |out|, with u_q = u_p = 2^-8 over a bf16 pool, 2^-11 over an
8-bit one (whose codes are exact). A bf16 weight or q may be an fp16 normal or not:
2^-24 absolute is below the 1e-5.
"""
import numpy as np
import pytest
import torch

import sink_window_attention_b200 as swa
from oracle import fp8, tokens

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 16, 16), (3, 5, 64, 48), (77, 12, 128, 128), (1000, 2, 128, 32),
                                       (5, 40, 256, 96)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("transpose", [False, True])
def test_rope(T, H, D, rot, layout, dtype, transpose):
    g = torch.Generator(device="cuda").manual_seed(T + rot)
    wide = torch.randn((T, H + 3, D), generator=g, device="cuda").to(dtype)
    x = wide[:, 1:H + 1]                                     # rows further apart than H * D
    pos = torch.randint(0, 2**31 - 1, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 2**31 - 1
    if T > 2:
        pos[1], pos[2] = 0, -5
    kw = dict(scale=0.25, original_len=4096.0)
    rope = swa.TokenRope(rot, layout=layout, amplitude=1.25, **kw)
    got = swa.token_rope_apply(x, pos, rope, transpose=transpose)
    # far positions: the angle in the table's own units (the turn per position is rounded to 2^-53 of itself)
    turns = np.array([t for t in rope.to_c().turns][:rot // 2], dtype=object)
    p = pos.cpu().numpy()
    want = np.zeros((T, H, D))
    xs = f64(x)
    for t in range(T):
        frac = np.array([float((int(p[t]) * int(w)) % 2**64) / 2.0**64 for w in turns])
        want[t] = tokens.rotate(xs[t:t + 1], [1], 2 * np.pi * frac, layout, 1.25, transpose)[0]
    mag = np.zeros_like(xs)
    a = np.abs(xs)
    n = rot // 2
    if layout == "half":
        mag[..., :n] = mag[..., n:rot] = a[..., :n] + a[..., n:rot]
    else:
        mag[..., 0:rot:2] = mag[..., 1:rot:2] = a[..., 0:rot:2] + a[..., 1:rot:2]
    u = 2.0**-8 if dtype == torch.bfloat16 else 2.0**-24
    assert np.all(np.abs(f64(got) - want) <= 1.25e-6 * mag + u * np.abs(want))
    # in place, with a stride
    assert torch.equal(swa.token_rope_apply(x, pos, rope, transpose=transpose, out=x), got)
    assert torch.equal(wide[:, 1:H + 1], got)


def test_rope_frequencies_at_ordinary_positions():
    """Against the definition's angles: 1e-14 of the angle's turns, below fp32's."""
    x = torch.randn((50, 3, 128), device="cuda")
    pos = i32(np.arange(50) * 41)
    for kw in (dict(), dict(scale=0.125, original_len=1024.0, theta0=500000.0)):
        got = swa.token_rope_apply(x, pos, swa.TokenRope(128, layout="half", **kw))
        want = tokens.rotate(f64(x), pos.cpu().numpy(), tokens.frequencies(128, **kw), "half")
        assert np.abs(f64(got) - want).max() <= 2e-6 * float(x.abs().max())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient(layout):
    """transpose=True is the gradient: against differences of y . R(x), which is linear
    in x (a step of 1 is exact but for fp32 rounding of the sum's terms), and R^T R = A^2."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x, y = (torch.randn((7, 3, 64), generator=g, device="cuda") for _ in range(2))
    pos = i32([0, 1, 17, 4095, 100000, 7, 8])
    rope = swa.TokenRope(32, layout=layout, amplitude=1.5)
    grad = f64(swa.token_rope_apply(y, pos, rope, transpose=True))
    base = f64(swa.token_rope_apply(x, pos, rope))
    for d in range(64):
        step = x.clone()
        step[:, :, d] += 1.0
        moved = f64(step[:, :, d]) - f64(x[:, :, d])
        diff = np.sum((f64(swa.token_rope_apply(step, pos, rope)) - base) * f64(y), axis=-1)
        assert np.abs(diff - grad[:, :, d] * moved).max() <= 64 * 4 * 1.5e-6
    back = swa.token_rope_apply(swa.token_rope_apply(x, pos, rope), pos, rope, transpose=True)
    want = x.clone()
    want[..., :32] *= 2.25
    assert (back - want).abs().max().item() <= 2e-5


def test_rope_of_no_tokens():
    x = torch.zeros((0, 4, 64), device="cuda")
    assert swa.token_rope_apply(x, i32([]), swa.TokenRope(64)).shape == (0, 4, 64)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
class Setup:
    """A ragged batch over a pool whose pages are in random order, and the oracle's copy."""

    def __init__(self, lens, news, H, D, dtype, page, seed=0, spare=2, garbage=False):
        r = np.random.default_rng(seed)
        self.lens, self.news, self.page, self.H, self.D, self.dtype = lens, news, page, H, D, dtype
        pages = [-(-n // page) for n in lens]
        n_pages = sum(pages) + spare
        order = r.permutation(n_pages)
        self.table = np.full((len(lens), max(1, max(pages)) + 1), -1, dtype=np.int64)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = swa.PagedKVCache(n_pages, page, H, D, dtype)
        self.pool = tokens.Pool(n_pages, page, H, D, dtype)
        self.start = np.concatenate([[0], np.cumsum(news)])
        if garbage:  # what an allocator hands out: NaN wherever nothing is written
            for name in ("k", "v", "k_scale", "v_scale"):
                t = getattr(self.cache, name)
                if t is not None:
                    t.fill_(0x7F if t.dtype == torch.uint8 else float("nan"))

    def batch(self, lens=None, news=None, table=None):
        lens = self.lens if lens is None else lens
        news = self.news if news is None else news
        return swa.TokenBatch(i32(np.concatenate([[0], np.cumsum(news)])), i32(lens),
                              i32(self.table if table is None else table), max(1, max(news)), max(1, max(lens)))

    def fill(self, seed):
        """Every token of every sequence in one append; returns k and v (rotated) per sequence."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = sum(self.lens)
        k = torch.randn((n, self.H, self.D), generator=g, device="cuda").bfloat16()
        v = torch.randn((n, self.H, self.D), generator=g, device="cuda").bfloat16()
        swa.paged_append(self.cache, self.batch(news=self.lens), k, v)
        self.take()

    def take(self):
        """The oracle's pool gets what the GPU's holds."""
        for name in ("k", "v"):
            t = getattr(self.cache, name)
            x = fp8.e4m3_decode_array(t.cpu().numpy()) if self.dtype == "fp8" else f64(t)
            setattr(self.pool, name, x)
            if self.dtype == "fp8":
                setattr(self.pool, name + "s", f64(getattr(self.cache, name + "_scale")))

    def keys(self, b, which, table=None):
        """[len][H][D] of sequence b, and which of its keys are in mapped pages."""
        table = self.table if table is None else table
        x = self.pool.values(which)
        n = self.lens[b]
        out, there = np.zeros((n, self.H, self.D)), np.zeros(n, dtype=bool)
        for j in range(n):
            p = table[b, j // self.page]
            if 0 <= p < self.pool.n_pages:
                out[j], there[j] = x[p, :, j % self.page], True
        return out, there


APPENDS = [  # (lengths before, new tokens, H, D, page)
    ([0], [1], 1, 64, 16),
    ([15, 16, 31, 0, 5], [1, 1, 1, 0, 1], 2, 128, 16),
    ([0, 7, 40], [33, 90, 1], 3, 128, 32),
    ([3, 100], [200, 28], 12, 64, 64),
    ([120, 1, 0], [9, 300, 127], 5, 128, 128),
    ([1], [130], 2, 64, 128),
]


@pytest.mark.parametrize("before,new,H,D,page", APPENDS)
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("layout", ["half", "interleaved", None])
def test_append(before, new, H, D, page, dtype, layout):
    lens = [a + b for a, b in zip(before, new)]
    s = Setup(lens, new, H, D, dtype, page, seed=page)
    rope = None if layout is None else swa.TokenRope(48, layout=layout)
    g = torch.Generator(device="cuda").manual_seed(9)

    def rows(news, grow):
        n = sum(news)
        wide = torch.randn((n + 2, 3 * H, D), generator=g, device="cuda").bfloat16() * grow
        return wide[:n, H:2 * H], wide[:n, 2 * H:]

    written = set()

    def run(lens_, news, grow):
        k, v = rows(news, grow)
        swa.paged_append(s.cache, s.batch(lens_, news), k, v, rope)
        at = 0
        for b, n in enumerate(news):
            pos = np.arange(lens_[b] - n, lens_[b])
            kk = f64(k[at:at + n])
            if rope is not None:
                kk = tokens.rotate(kk, pos, tokens.frequencies(48), layout)
            s.pool.append(list(s.table[b]), lens_[b], kk, f64(v[at:at + n]))
            written.update((s.table[b, p // page], p % page) for p in pos)
            at += n

    if sum(before):
        run(before, before, 1.0)
    run(lens, new, 1.7)  # larger values: the scales of pages that hold older tokens grow
    mask = np.zeros((s.pool.n_pages, 1, page, 1), dtype=bool)
    for p, r in written:
        mask[p, 0, r] = True
    for name in ("k", "v"):
        t, want = getattr(s.cache, name), s.pool.values(name)
        if dtype == "bf16":
            got = f64(t)
            # K: rounded once after an fp32 rotation of elements below 2 * 1.7 * 6
            assert np.all(np.abs(got - want) <= 2.0**-8 * np.abs(want) + 3e-5)
            if name == "v" or rope is None:
                assert np.array_equal(got, want)
        else:
            sc = f64(getattr(s.cache, name + "_scale"))
            assert np.array_equal(sc, getattr(s.pool, name + "s")), name
            got = fp8.e4m3_decode_array(t.cpu().numpy()) * sc[..., None, None]
            # equal codes, but where the fp32 rotation falls on the other side of a border:
            # one step, 2^-3 of the value (2^-9 of the scale below the normals), and rarely
            off = np.abs(got - want)
            assert np.all(off <= 2.0**-3 * np.abs(want) * 1.01 + 2.0**-9 * sc[..., None, None])
            if name == "v" or rope is None:
                assert np.array_equal(got, want)
            assert np.mean(off > 0) <= 1e-3
        assert np.all(got[~np.broadcast_to(mask, got.shape)] == 0)  # nothing else was touched


def test_append_token_by_token_equals_one_call():
    """bf16: the same bits. 8-bit: the same scale, and the same codes but below the normals."""
    for dtype in ("bf16", "fp8"):
        a, b = (Setup([70], [70], 3, 64, dtype, 32, seed=1) for _ in range(2))
        g = torch.Generator(device="cuda").manual_seed(2)
        k = torch.randn((70, 3, 64), generator=g, device="cuda")
        k = (k * torch.exp2(torch.arange(70, device="cuda") / 8.0)[:, None, None]).bfloat16()
        rope = swa.TokenRope(64)
        swa.paged_append(a.cache, a.batch(), k, k, rope)
        for t in range(70):
            swa.paged_append(b.cache, b.batch([t + 1], [1]), k[t:t + 1], k[t:t + 1], rope)
        if dtype == "bf16":
            assert torch.equal(a.cache.k, b.cache.k) and torch.equal(a.cache.v, b.cache.v)
            continue
        assert torch.equal(a.cache.k_scale, b.cache.k_scale) and torch.equal(a.cache.v_scale, b.cache.v_scale)
        for x, y in ((a.cache.k, b.cache.k), (a.cache.v, b.cache.v)):
            x, y = x.view(torch.float8_e4m3fn).float(), y.view(torch.float8_e4m3fn).float()
            assert torch.equal(x[x.abs() >= 2.0**-6], y[x.abs() >= 2.0**-6])
            assert (x - y).abs().max().item() <= 2.0**-9


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_append_where_no_page_is_mapped_and_rows_of_no_sequence(dtype):
    """Tokens whose page entry names no page are dropped; rows behind the last
    sequence and positions before 0 are not written; the rest is."""
    s = Setup([40, 20], [40, 20], 2, 64, dtype, 16)
    table = s.table.copy()
    table[0, 1], table[1, 0] = s.pool.n_pages, -7
    k = torch.randn((64, 2, 64), device="cuda").bfloat16()
    t = i32(table)
    swa.paged_append(s.cache, swa.TokenBatch(i32([0, 40, 60]), i32([40, 20]), t, 40, 40), k, k)
    for b, n, at in ((0, 40, 0), (1, 20, 40)):
        s.pool.append(list(table[b]), n, f64(k[at:at + n]), f64(k[at:at + n]))
    def held():
        return fp8.e4m3_decode_array(s.cache.v.cpu().numpy()) * f64(s.cache.v_scale)[..., None, None] \
            if dtype == "fp8" else f64(s.cache.v)
    assert np.array_equal(held(), s.pool.values("v"))
    # 8 rows for a sequence of 5 tokens: the first three stand before position 0
    fresh = Setup([5], [8], 2, 64, dtype, 16)
    swa.paged_append(fresh.cache, fresh.batch([5], [8]), k[:8], k[:8])
    fresh.pool.append(list(fresh.table[0]), 5, f64(k[3:8]), f64(k[3:8]))
    s = fresh
    assert np.array_equal(held(), s.pool.values("v"))


def test_append_of_non_finite_values():
    """Infinities saturate at the scale the finite values ask for, NaN stays NaN."""
    s = Setup([16], [16], 1, 64, "fp8", 16)
    k = torch.randn((16, 1, 64), device="cuda").bfloat16()
    k[3, 0, 5], k[4, 0, 6], k[5, 0, 7] = float("inf"), float("-inf"), float("nan")
    swa.paged_append(s.cache, s.batch(), k, k)
    p = int(s.table[0, 0])
    amax = float(k[torch.isfinite(k)].abs().max())
    assert s.cache.v_scale[p, 0].item() == tokens.two_power_scale(amax)
    x = s.cache.v.view(torch.float8_e4m3fn).float()[p, 0]
    assert x[3, 5].item() == 448 and x[4, 6].item() == -448 and torch.isnan(x[5, 7])
    assert torch.isnan(x).sum().item() == 1


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def check(s, q, got, lse, *, rope=None, table=None, scores=None, untouched=None):
    """Every row against the oracle, with the header's elementwise bound."""
    kw = scores or {}
    u = 2.0**-11 if s.dtype == "fp8" else 2.0**-8
    got, lse = f64(got), f64(lse)
    qs = f64(q)
    at = 0
    for b, n in enumerate(s.news):
        if n == 0:
            continue
        pos = np.arange(s.lens[b] - n, s.lens[b])
        x = qs[at:at + n]
        if rope is not None:
            x = tokens.rotate(x, pos, rope["w"], rope["layout"])
        (k, there), (v, _) = s.keys(b, "k", table), s.keys(b, "v", table)
        args = {**kw, "prefix": kw["prefix"][b]} if "prefix" in kw else kw
        out, ref_lse, mag, dots = tokens.attend(x, k, v, s.lens[b], exists=there, **args)
        cap = 1e-5 if kw.get("cap") else 0.0
        eps = (u + 2.0**-20) * dots + cap
        bound = (np.expm1(2 * eps) + u + 1e-5)[..., None] * mag + 2.0**-8 * np.abs(out)
        err = np.abs(got[at:at + n] - out)
        assert np.all(err <= bound), (b, float((err / np.maximum(bound, 1e-30)).max()))
        assert np.array_equal(np.isinf(lse[at:at + n]), np.isinf(ref_lse))
        fin = np.isfinite(ref_lse)
        assert np.all(np.abs(lse[at:at + n] - np.where(fin, ref_lse, 0))[fin] <= (eps + 1e-5 * (1 + np.abs(ref_lse)))[fin])
        # the roundings are independent, so the whole is far nearer than the worst case of each
        norm = np.linalg.norm(out)
        if norm > 0 and out.size >= 4096:
            assert np.linalg.norm(err) / norm <= 8e-3
        at += n


def attention(s, Hq, seed=4, rope=None, table=None, news=None, rows_behind=2, **scores):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = sum(s.news)
    wide = torch.randn((n + rows_behind, Hq + 5, s.D), generator=g, device="cuda").bfloat16()
    q = wide[:, 2:2 + Hq]
    out = torch.full((n + rows_behind, Hq, s.D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + rows_behind, Hq), 7.0, device="cuda")
    kw = dict(scores)
    sc = swa.Scores(softmax_scale=kw.get("scale", 0.0), window=kw.get("window", 0), n_sink=kw.get("n_sink", 0),
                    soft_cap=kw.get("cap", 0.0), slopes=kw.get("slopes"),
                    prefix_len=i32(kw["prefix"]) if "prefix" in kw else None)
    tr = None if rope is None else swa.TokenRope(rope["rot"], layout=rope["layout"])
    swa.paged_attention(q, s.cache, s.batch(table=table), tr, sc, out=out, lse=lse)
    assert swa.device_error() == 0
    assert torch.all(out[n:] == 7.0) and torch.all(lse[n:] == 7.0)  # rows of no sequence
    if rope is not None:
        rope = {**rope, "w": tokens.frequencies(rope["rot"])}
    check(s, q, out, lse, rope=rope, table=table, scores=scores)
    return q, out, lse


SHAPES = [  # (lengths, new tokens, H, group, D, page)
    ([1], [1], 1, 1, 64, 16),
    ([17, 16, 15, 0, 64], [1, 1, 1, 0, 1], 2, 4, 128, 16),
    ([700], [1], 2, 8, 128, 64),
    ([300, 45, 2], [5, 3, 2], 3, 3, 64, 32),
    ([5000, 33], [2, 1], 1, 7, 128, 128),
    ([260, 131, 77], [130, 131, 20], 2, 2, 128, 16),
    ([400, 90], [300, 90], 1, 1, 64, 16),
    ([1300], [257], 1, 5, 128, 32),
]
MODS = {
    "plain": {},
    "window": dict(window=37),
    "sink": dict(window=20, n_sink=3),
    "cap": dict(cap=2.0, scale=0.3),
    "bias": dict(bias=True),
    "all": dict(window=50, n_sink=18, cap=5.0, bias=True, prefix=True),
    "prefix": dict(prefix=True),
    "one": dict(window=1),
}


@pytest.mark.parametrize("lens,news,H,group,D,page", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("mod", list(MODS))
def test_attention(lens, news, H, group, D, page, dtype, mod):
    s = Setup(lens, news, H, D, dtype, page, seed=len(lens), garbage=True)
    s.fill(5)
    kw = dict(MODS[mod])
    if kw.pop("bias", False):
        kw["slopes"] = [float(2.0 ** (-1 - h)) for h in range(H * group)]
    if kw.pop("prefix", False):
        kw["prefix"] = [n // 2 + 1 if b % 2 == 0 else 0 for b, n in enumerate(lens)]
        kw["prefix"][-1] = max(kw["prefix"][-1], lens[-1] + 50)  # beyond the last key: all of them
    rope = dict(rot=64, layout="half") if mod == "plain" else dict(rot=32, layout="interleaved") if mod == "sink" else None
    attention(s, H * group, rope=rope, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("new", [1, 150])
def test_attention_over_pages_that_were_given_back(dtype, new):
    """A window over pages whose older neighbours are unmapped, and a row that sees
    no key at all: 0 and -inf."""
    s = Setup([420, 300], [new, new], 2, 64, dtype, 16, garbage=True)
    s.fill(6)
    table = s.table.copy()
    first = 420 - new
    table[0, 1:(first - 31) // 16] = -1     # neither sinks nor window reach these
    attention(s, 4, table=table, window=32, n_sink=9)
    table[1, :] = s.pool.n_pages + 5
    q, out, lse = attention(s, 4, table=table, window=32, n_sink=9)
    assert torch.all(out[new:2 * new] == 0) and torch.all(torch.isinf(lse[new:2 * new]))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_more_rows_than_keys(dtype):
    """Rows before position 0 see nothing."""
    for new in (12, 200):
        s = Setup([5, new + 3], [new, new], 2, 64, dtype, 16, garbage=True)
        s2 = Setup([5, new + 3], [5, new + 3], 2, 64, dtype, 16, garbage=True)
        s2.fill(8)
        s2.news = s.news
        q, out, lse = attention(s2, 2)
        assert torch.all(out[:new - 5] == 0) and torch.all(torch.isinf(lse[:new - 5]))


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 140])
def test_scales_far_apart_and_large_scores(dtype, D, new):
    """Pages whose values differ by powers of two (8-bit: scales 2^-20 to 2^20 apart),
    and queries large enough that the running maximum moves by hundreds."""
    s = Setup([700], [700], 2, D, dtype, 16, garbage=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((700, 2, D), generator=g, device="cuda")
    k = k * torch.linspace(0.1, 12, 700, device="cuda")[:, None, None]
    v = torch.randn((700, 2, D), generator=g, device="cuda")
    v = v * torch.exp2(((torch.arange(700, device="cuda") // 16) * 7 % 41 - 20).float())[:, None, None]
    swa.paged_append(s.cache, s.batch(), k.bfloat16(), v.bfloat16())
    s.take()
    s.news = [new]
    attention(s, 4)
    v[:] = 0  # zero pages: scale 0
    swa.paged_append(s.cache, s.batch([700], [700]), k.bfloat16(), v.bfloat16())
    out = swa.paged_attention(torch.randn((new, 4, D), device="cuda").bfloat16(), s.cache, s.batch([700], [new]))
    assert torch.all(out == 0)


@pytest.mark.parametrize("D,page", [(64, 32), (128, 16), (128, 128)])
@pytest.mark.parametrize("new", [1, 7, 140])
def test_scales_that_are_no_powers_of_two(D, page, new):
    """A pool that something else filled: any codes but NaN, any positive scales."""
    s = Setup([333, 150], [new, new], 2, D, "fp8", page)
    g = torch.Generator(device="cuda").manual_seed(new)
    for name in ("k", "v"):
        codes = torch.randint(0, 127, s.cache.k.shape, generator=g, device="cuda") + \
            128 * torch.randint(0, 2, s.cache.k.shape, generator=g, device="cuda")
        getattr(s.cache, name).copy_(codes.to(torch.uint8))
        getattr(s.cache, name + "_scale").copy_(0.003 + 0.01 * torch.rand(s.cache.k.shape[:2], generator=g, device="cuda"))
    s.take()
    # rounding V's code times the scale's mantissa to fp16 is the bound's weight rounding once more
    attention(s, 8)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_many_sequences_and_many_heads(dtype):
    """300 sequences of 0 to 40 tokens; 128 query heads on one K/V head."""
    r = np.random.default_rng(5)
    lens = [int(n) for n in r.integers(0, 41, 300)]
    s = Setup(lens, [min(1, n) for n in lens], 1, 64, dtype, 16, garbage=True)
    s.fill(2)
    attention(s, 3, window=9, n_sink=2)
    for new in (1, 3):
        s = Setup([90], [new], 1, 128, dtype, 32, garbage=True)
        s.fill(3)
        attention(s, 128, slopes=[0.01 * h for h in range(128)])


def test_calls_from_two_threads():
    """One batch and cache, two threads with row counts of their own."""
    import threading
    s = Setup([500, 400], [1, 1], 2, 64, "fp8", 16)
    s.fill(2)
    b = s.batch()
    qs = [torch.randn((n, 4, 64), device="cuda").bfloat16() for n in (2, 5)]
    want = [swa.paged_attention(q, s.cache, b)[:2].clone() for q in qs]
    bad = []

    def work(q, w):
        st = torch.cuda.Stream()
        for _ in range(50):
            with torch.cuda.stream(st):
                got = swa.paged_attention(q, s.cache, b)
                st.synchronize()
                if not torch.equal(got[:2], w):
                    bad.append(1)

    torch.cuda.synchronize()
    ts = [threading.Thread(target=work, args=a) for a in zip(qs, want)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_bounds_of_the_host_hold_on_the_device():
    """Arrays that say more than the host's bounds: rows beyond max_q and total_q are
    not processed, keys beyond max_kv and the table do not exist."""
    s = Setup([64], [4], 1, 64, "bf16", 16)
    s.fill(3)
    q = torch.randn((4, 1, 64), device="cuda").bfloat16()
    want = swa.paged_attention(q, s.cache, s.batch())
    out = torch.full((4, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    t = i32(s.table[:, :4])
    swa.paged_attention(q, s.cache, swa.TokenBatch(i32([0, 4]), i32([64]), t, 2, 64), out=out)
    assert torch.equal(out[:2], want[:2]) and torch.all(out[2:] == 5.0)
    # q_start past the rows, a length past table and bound
    out.fill_(5.0)
    swa.paged_attention(q, s.cache, swa.TokenBatch(i32([2, 1000]), i32([1 << 30]), t, 1000, 1 << 30), out=out)
    assert torch.all(out[:2] == 5.0) and torch.isfinite(out).all()
    out.fill_(5.0)
    swa.paged_attention(q, s.cache, swa.TokenBatch(i32([3, 1]), i32([-4]), t, 4, 64), out=out)
    assert torch.all(out == 5.0)
    k = torch.randn((4, 1, 64), device="cuda").bfloat16()
    before = s.cache.k.clone()
    swa.paged_append(s.cache, swa.TokenBatch(i32([0, 4]), i32([1 << 30]), t, 4, 64), k, k)
    assert torch.equal(before, s.cache.k)
    assert swa.device_error() == 0


# ---------------------------------------------------------------------------
# the path as it is used
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_stream_of_steps(dtype):
    """Prompts, then tokens one at a time through append and attention, against an
    oracle that keeps every token's bf16 key and value: over a bf16 pool the header's
    bound; over an 8-bit pool K and V carry one rounding of 2^-4 more."""
    H, group, D, page = 2, 3, 64, 16
    prompts = [37, 5, 16]
    steps = 20
    lens = [p + steps for p in prompts]
    s = Setup(lens, [1] * 3, H, D, dtype, page, garbage=True)
    rope = swa.TokenRope(64, layout="half")
    w = tokens.frequencies(64)
    g = torch.Generator(device="cuda").manual_seed(11)
    table = i32(s.table)
    keys = [[np.zeros((0, H, D)), np.zeros((0, H, D))] for _ in lens]
    now = [0, 0, 0]
    for step in range(steps + 1):
        new = prompts if step == 0 else [1, 1, 1]
        now = [a + b for a, b in zip(now, new)]
        qkv = torch.randn((sum(new), (group + 2) * H, D), generator=g, device="cuda").bfloat16()
        q, k, v = qkv[:, :group * H], qkv[:, group * H:(group + 1) * H], qkv[:, (group + 1) * H:]
        batch = swa.TokenBatch(i32(np.concatenate([[0], np.cumsum(new)])), i32(now), table, max(new), max(now))
        swa.paged_append(s.cache, batch, k, v, rope)
        out = f64(swa.paged_attention(q, s.cache, batch, rope, swa.Scores(window=30, n_sink=4)))
        at = 0
        for b, n in enumerate(new):
            pos = np.arange(now[b] - n, now[b])
            kk = tokens.rotate(f64(k[at:at + n]), pos, w, "half")
            keys[b] = [np.concatenate([keys[b][0], kk]), np.concatenate([keys[b][1], f64(v[at:at + n])])]
            qq = tokens.rotate(f64(q[at:at + n]), pos, w, "half")
            ref, _, mag, dots = tokens.attend(qq, keys[b][0], keys[b][1], now[b], window=30, n_sink=4)
            uk, uv = (2.0**-4, 2.0**-4) if dtype == "fp8" else (2.0**-8, 0.0)
            eps = (2.0**-8 + uk) * dots
            bound = (np.expm1(2 * eps) + 2.0**-8 + uv + 1e-5)[..., None] * mag + 2.0**-8 * np.abs(ref)
            assert np.all(np.abs(out[at:at + n] - ref) <= bound), (step, b)
            at += n
    assert swa.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("new", [1, 40])
def test_captured_and_replayed_on_other_streams(dtype, new):
    """append + attention captured once and replayed with other lengths, tokens and
    pages, two graphs that share a workspace replayed in turn, and the same call on a
    side stream: the bits of the eager call."""
    s = Setup([2000, 900], [new, new], 2, 64, dtype, 16)
    s.fill(1)
    rope = swa.TokenRope(64)
    start, table = i32([0, new, 2 * new]), i32(s.table)
    lens = i32([2000, 900])
    batch = swa.TokenBatch(start, lens, table, new, 2000)
    qkv = torch.randn((2 * new, 8, 64), device="cuda").bfloat16()
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    n = swa.paged_attention_workspace_bytes(s.cache, batch, 2 * new, 4)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")

    def step(**kw):
        swa.paged_append(s.cache, batch, k, v, rope, **kw)
        return swa.paged_attention(q, s.cache, batch, rope, workspace=ws, **kw)

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step()
        graphs.append((gr, out))
    for now in ([2000, 900], [1990, 800], [new, 899]):
        lens.copy_(i32(now))
        qkv.normal_()
        eager = step().clone()
        for gr, out in graphs + graphs[::-1]:
            gr.replay()
            assert torch.equal(out, eager)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = step(stream=side)
        fresh = swa.paged_attention(q, s.cache, batch, rope, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(other, eager) and torch.equal(fresh, eager)
    assert swa.device_error() == 0


def test_two_calls_at_once_on_two_streams():
    """Without a workspace each call has its own scratch: two streams at once give the
    bits of one after the other."""
    s = Setup([3001, 2500], [1, 1], 2, 128, "fp8", 16)
    s.fill(2)
    b = s.batch()
    qs = [torch.randn((2, 16, 128), device="cuda").bfloat16() for _ in range(2)]
    want = [swa.paged_attention(q, s.cache, b) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [swa.paged_attention(q, s.cache, b, stream=st) for q, st in zip(qs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes for K: the pages at its end are written and read."""
    page, H, D = 128, 16, 128
    n_pages = 2**32 // (page * H * D * 2) + 40
    cache = swa.PagedKVCache(n_pages, page, H, D, "bf16")
    table = i32([[n_pages - 1, 3, n_pages - 2]])
    k = torch.randn((300, H, D), device="cuda").bfloat16()
    batch = swa.TokenBatch(i32([0, 300]), i32([300]), table, 300, 300)
    swa.paged_append(cache, batch, k, k)
    assert torch.equal(cache.k[n_pages - 1], k[:128].transpose(0, 1))
    assert torch.equal(cache.v[n_pages - 2, :, :44], k[256:].transpose(0, 1))
    small = swa.PagedKVCache(4, page, H, D, "bf16")
    t2 = i32([[2, 0, 1]])
    b2 = swa.TokenBatch(i32([0, 300]), i32([300]), t2, 300, 300)
    swa.paged_append(small, b2, k, k)
    for new in (300, 1):
        q = torch.randn((new, 2 * H, D), device="cuda").bfloat16()
        got = swa.paged_attention(q, cache, swa.TokenBatch(i32([0, new]), i32([300]), table, new, 300))
        want = swa.paged_attention(q, small, swa.TokenBatch(i32([0, new]), i32([300]), t2, new, 300))
        assert torch.equal(got, want)
