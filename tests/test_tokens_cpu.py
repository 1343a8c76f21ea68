"""Token streams without a GPU: the frequency table, the oracle's own pins, and
the refusals of every entry point (all on the host, before anything is launched)."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import sink_window_attention_b200 as swa
from oracle import tokens
from tests.conftest import ROOT


@pytest.fixture(scope="module")
def L():
    from sink_window_attention_b200 import build
    build.build()
    return swa.lib()


def test_struct_layouts_match_the_header(tmp_path):
    structs = (("ll_token_rope_desc", swa.TokenRopeDescC), ("ll_paged_cache", swa.PagedCacheC),
               ("ll_token_batch", swa.TokenBatchC), ("ll_score_desc", swa.ScoreDescC))
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "ll_api.h"', "int main(void) {"]
    for cname, cls in structs:
        lines.append(f'  printf("{cname} sizeof %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "l.c").write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o",
                    str(tmp_path / "l")], check=True)
    got = {}
    for line in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.splitlines():
        s, f, v = line.split()
        got[(s, f)] = int(v)
    for cname, cls in structs:
        assert got[(cname, "sizeof")] == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert got[(cname, f)] == getattr(cls, f).offset, (cname, f)
    header = open(os.path.join(ROOT, "include", "ll_api.h")).read()
    assert f"#define LL_MAX_TOKEN_HEADS {swa.MAX_TOKEN_HEADS}" in header
    assert f"#define LL_MAX_TOKEN_PAIRS {swa.MAX_TOKEN_PAIRS}" in header


@pytest.mark.parametrize("kw", [dict(), dict(theta0=500000.0), dict(scale=0.25), dict(scale=0.25, original_len=4096),
                                dict(scale=0.125, original_len=32768, beta_fast=16.0, beta_slow=0.5)])
@pytest.mark.parametrize("rot", [16, 48, 96, 128])
def test_turn_table(L, rot, kw):
    """turns[i] / 2^64 is w_i / (2 pi) to the last bits of a double."""
    r = swa.TokenRope(rot, **kw).to_c()
    w = tokens.frequencies(rot, **kw)
    got = np.array([t / 2.0 ** 64 for t in r.turns])
    assert np.all(got[rot // 2:] == 0)
    assert np.allclose(got[:rot // 2] * 2 * math.pi, w, rtol=1e-14, atol=1e-18)


def test_oracle_scale_is_the_smallest_power_of_two():
    for a in [1e-30, 0.1, 1.0, 447.9, 448.0, 448.1, 3.5, 1.75, 1.7500001, 3e38]:
        s = tokens.two_power_scale(a)
        assert 448 * s >= a and (448 * s / 2 < a) and math.log2(s) == round(math.log2(s))
    assert tokens.two_power_scale(0.0) == 0.0


def test_oracle_rotation_pins():
    """Position 1 of pair 0 turns by one radian; the transpose undoes it; scores
    depend on the difference of positions alone."""
    w = tokens.frequencies(16)
    x = np.zeros((1, 1, 32))
    x[0, 0, 0] = 1.0
    assert np.allclose(tokens.rotate(x, [1], w, "half")[0, 0, [0, 8]], [math.cos(1), math.sin(1)])
    assert np.allclose(tokens.rotate(x, [1], w, "interleaved")[0, 0, [0, 1]], [math.cos(1), math.sin(1)])
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(2, 1, 1, 32))
    for layout in ("half", "interleaved"):
        y = tokens.rotate(tokens.rotate(q, [77], w, layout), [77], w, layout, transpose=True)
        assert np.allclose(y, q)
        d = [np.sum(tokens.rotate(q, [a], w, layout) * tokens.rotate(k, [b], w, layout)) for a, b in ((9, 4), (105, 100))]
        assert np.allclose(*d)


def test_oracle_append_token_by_token_carries_one_rounding():
    """Powers of two make the re-coding exact, so a page filled token by token holds
    what one call writes, but for codes that underflow."""
    rng = np.random.default_rng(1)
    x = rng.normal(size=(16, 1, 32)) * np.exp2(np.arange(16) / 3)[:, None, None]
    a, b = tokens.Pool(1, 16, 1, 32, "fp8"), tokens.Pool(1, 16, 1, 32, "fp8")
    a.append([0], 16, x, x)
    for t in range(16):
        b.append([0], t + 1, x[t:t + 1], x[t:t + 1])
    assert a.ks[0, 0] == b.ks[0, 0]
    av, bv = a.values("k"), b.values("k")
    normal = np.abs(av) >= 2.0 ** -6 * a.ks[0, 0]
    assert np.array_equal(av[normal], bv[normal])
    assert np.all(np.abs(av - bv) <= 2.0 ** -9 * a.ks[0, 0])


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
A = 1 << 20  # a well aligned address that is never dereferenced on these paths


def _cache(**kw):
    c = swa.PagedCacheC(A, 2 * A, None, None, swa.LL_BF16, 100, 16, 8, 128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _fp8(**kw):
    return _cache(**{**dict(dtype=swa.LL_FP8_E4M3, k_scale=3 * A, v_scale=4 * A), **kw})


def _batch(**kw):
    t = swa.TokenBatchC(5 * A, 6 * A, 7 * A, 4, 64, 4, 1, 1000)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _rope(**kw):
    r = swa.TokenRope(64).to_c()
    for k, v in kw.items():
        setattr(r, k, v)
    return r


CACHES = [(dict(k=None), "NULL"), (dict(v=A + 8), "aligned"), (dict(dtype=swa.LL_F32), "dtype"),
          (dict(dtype=swa.LL_FP8_E4M3), "k_scale"), (dict(dtype=swa.LL_FP8_E4M3, k_scale=A + 2, v_scale=A), "4-byte"),
          (dict(n_pages=0), "positive"), (dict(H=0), "positive"), (dict(page_size=24), "page_size"),
          (dict(page_size=256), "page_size"), (dict(page_size=0), "page_size"), (dict(D=96), "D = 96"),
          (dict(H=129), "exceeds")]
BATCHES = [(dict(q_start=None), "NULL"), (dict(kv_len=None), "NULL"), (dict(page_table=None), "NULL"),
           (dict(kv_len=A + 2), "aligned"), (dict(B=0), "positive"), (dict(max_pages=0), "positive"),
           (dict(B=65536), "65535"), (dict(total_q=-1), ">= 0"), (dict(max_q=-1), ">= 0"), (dict(max_kv=-1), ">= 0")]
ROPES = [(dict(rot_dim=0), "rot_dim"), (dict(rot_dim=24), "rot_dim"), (dict(rot_dim=144), "rot_dim"),
         (dict(layout=2), "layout"), (dict(amplitude=float("nan")), "amplitude")]


def _attend(L, cache=None, batch=None, rope=None, scores=None, q=A, stride=32 * 128, dt=swa.LL_BF16, Hq=32, out=A,
            lse=None, ws=A, ws_bytes=1 << 40):
    return L.ll_paged_attention(q, stride, dt, Hq, cache or _cache(), batch or _batch(), rope, scores, out, lse, ws,
                                ws_bytes, None)


def _append(L, cache=None, batch=None, rope=None, k=A, ks=1024, v=A, vs=1024, dt=swa.LL_BF16):
    return L.ll_paged_append(cache or _cache(), batch or _batch(), k, ks, v, vs, dt, rope, None)


def refused(L, st, msg, want=swa.LL_ERR_INVALID_ARG):
    assert st == want, (st, swa.last_error())
    assert msg in swa.last_error(), swa.last_error()


@pytest.mark.parametrize("call", [_attend, _append])
def test_descriptor_refusals(L, call):
    for kw, msg in CACHES:
        refused(L, call(L, cache=_cache(**kw)), msg)
    for kw, msg in BATCHES:
        refused(L, call(L, batch=_batch(**kw)), msg)
    for kw, msg in ROPES:
        refused(L, call(L, rope=_rope(**kw)), msg)
    narrow = dict(cache=_cache(D=64), rope=_rope(rot_dim=96))
    refused(L, call(L, **narrow, **({} if call is _append else dict(stride=32 * 64))), "rot_dim")


def test_append_refusals(L):
    for kw, msg in [(dict(k=None), "k must"), (dict(v=None), "v must"), (dict(k=A + 2), "aligned"),
                    (dict(ks=1023), "stride"), (dict(vs=1016), "stride"), (dict(dt=swa.LL_F32), "BF16")]:
        refused(L, _append(L, **kw), msg)


def test_attention_refusals(L):
    sc = swa.ScoreDescC
    long = _batch(max_kv=200000, max_pages=20000)  # its pieces are joined through the workspace
    bad = (ctypes.c_float * 32)(*([0.0] * 31 + [float("inf")]))
    slopes = sc()
    slopes.slopes = ctypes.cast(bad, ctypes.POINTER(ctypes.c_float))
    for kw, msg in [(dict(q=None), "q must"), (dict(q=A + 8), "aligned"), (dict(out=None), "out"),
                    (dict(out=A + 4), "out"), (dict(lse=A + 2), "lse"), (dict(stride=32 * 128 - 8), "stride"),
                    (dict(stride=32 * 128 + 4), "stride"), (dict(dt=swa.LL_F32), "BF16"), (dict(Hq=12), "multiple"),
                    (dict(Hq=0), "multiple"), (dict(scores=sc(-1.0)), "softmax_scale"),
                    (dict(scores=sc(float("inf"))), "softmax_scale"), (dict(scores=sc(0.0, -2.0)), "soft_cap"),
                    (dict(scores=sc(0.0, float("nan"))), "soft_cap"),
                    (dict(scores=sc(0.0, 1e-44)), "range"), (dict(scores=sc(3e38)), "range"), (dict(scores=sc(0.0, 0.0, -1)), "window"),
                    (dict(scores=sc(0.0, 0.0, 0, -1)), "n_sink"), (dict(scores=sc(0.0, 0.0, 0, 0, A + 2)), "prefix_len"),
                    (dict(scores=slopes), "slopes[31]"), (dict(batch=long, ws_bytes=16), "workspace"),
                    (dict(batch=long, ws=None), "workspace"), (dict(batch=long, ws=A + 4), "workspace")]:
        refused(L, _attend(L, **kw), msg)
    refused(L, _attend(L, Hq=136, stride=136 * 128), "exceeds", swa.LL_ERR_UNSUPPORTED)


def test_rope_refusals(L):
    def apply(x=A, xs=1024, out=A, os_=1024, dt=swa.LL_BF16, pos=A, T=3, H=8, D=128, rope=None, null=False):
        return L.ll_token_rope_apply(x, xs, out, os_, dt, pos, T, H, D, None if null else (rope or _rope()), 0, None)
    for kw, msg in [(dict(x=None), "x must"), (dict(out=None), "out must"), (dict(x=A + 2), "aligned"),
                    (dict(xs=1000), "stride"), (dict(os_=1028), "stride"), (dict(dt=swa.LL_FP8_E4M3), "dtype"),
                    (dict(pos=None), "positions"), (dict(pos=A + 1), "positions"), (dict(T=-1), "T >= 0"),
                    (dict(H=0), "H >= 1"), (dict(D=120), "multiple of 16"), (dict(null=True), "rope")]:
        refused(L, apply(**kw), msg)
    for kw, msg in ROPES:
        refused(L, apply(rope=_rope(**kw)), msg)
    refused(L, apply(D=48, xs=8 * 48, os_=8 * 48), "rot_dim")
    refused(L, apply(D=2048, xs=8 * 2048, os_=8 * 2048), "1024", swa.LL_ERR_UNSUPPORTED)
    for kw, msg in [(dict(rot_dim=0), "rot_dim"), (dict(rot_dim=130), "rot_dim"), (dict(theta0=1.0), "theta0"),
                    (dict(theta0=float("nan")), "theta0"), (dict(scale=0.0), "scale"), (dict(scale=1.5), "scale"),
                    (dict(original_len=-1.0), "original_len"), (dict(original_len=64, beta_fast=1.0), "beta"),
                    (dict(amplitude=float("inf")), "amplitude")]:
        with pytest.raises(swa.LLError) as e:
            swa.TokenRope(**{**dict(rot_dim=64), **kw})
        assert e.value.status == swa.LL_ERR_INVALID_ARG and msg in str(e.value)
    with pytest.raises(ValueError, match="layout"):
        swa.TokenRope(64, layout="neox")


def test_workspace_is_zero_for_short_histories_and_bad_descriptors(L):
    ws = L.ll_paged_attention_workspace_bytes
    assert ws(_cache(), _batch(max_kv=256), 32) == 0
    assert ws(_cache(), _batch(max_kv=200000, max_pages=20000), 32) > 0
    assert ws(_cache(), _batch(total_q=0), 32) == 0
    assert ws(_cache(D=96), _batch(), 32) == 0 and ws(_cache(), _batch(B=0), 32) == 0 and ws(_cache(), _batch(), 12) == 0


def test_pool_bound_and_kept_descriptors(L):
    refused(L, _append(L, cache=_cache(n_pages=1 << 29, H=8)), "2^31 - 1")
    import torch
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    batch = swa.TokenBatch(i32(3), i32(2), i32(2, 4), 1, 64)
    cache = swa.PagedKVCache(4, 16, 2, 64, "fp8", device="cpu")
    a = cache.to_c()
    assert cache.to_c() is a and (a.n_pages, a.page_size, a.H, a.D, a.dtype) == (4, 16, 2, 64, swa.LL_FP8_E4M3)
    cache.k = cache.k.clone()  # another tensor: another descriptor, the old one left as it was
    b = cache.to_c()
    assert b is not a and b.k == cache.k.data_ptr() and a.k != b.k and b.v == a.v
    with pytest.raises(ValueError, match="CUDA"):
        batch.to_c(2, 0)


def test_binding_refusals(L):
    import torch
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    cache = swa.PagedKVCache(4, 16, 2, 64, device="cpu")
    batch = swa.TokenBatch(i32(3), i32(2), i32(2, 4), 1, 64)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        swa.paged_append(cache, batch, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        swa.paged_attention(x, cache, batch)
    with pytest.raises(ValueError, match="CUDA"):
        swa.token_rope_apply(x, i32(2), swa.TokenRope(64))
    with pytest.raises(ValueError, match="k must be"):
        swa.paged_append(cache, batch, x[:, :1], x)
    with pytest.raises(ValueError, match="contiguous"):
        swa.paged_append(cache, batch, torch.zeros(2, 64, 2, dtype=torch.bfloat16).transpose(1, 2), x)
    with pytest.raises(ValueError, match="q_start"):
        swa.TokenBatch(i32(2), i32(2), i32(2, 4), 1, 64)
    with pytest.raises(ValueError, match="kv_len"):
        swa.TokenBatch(i32(3), i32(2).long(), i32(2, 4), 1, 64)
    with pytest.raises(ValueError, match="page_table"):
        swa.TokenBatch(i32(3), i32(2), i32(8), 1, 64)
    with pytest.raises(ValueError, match="slopes"):
        swa.Scores(slopes=[0.5] * 3).to_c(2, 4)
    with pytest.raises(ValueError, match="prefix_len"):
        swa.Scores(prefix_len=i32(3)).to_c(2, 4)
