"""The norm check of attention over a paged pool tells a right output from a wrong one,
whatever the shape: zeros, a piece of the keys left out, pieces joined at equal weight."""
import numpy as np
import pytest
import torch

from oracle import tokens
from tests.paged_checks import norm_error, norm_limit
from tests.test_gpu_paged_numerics import LONG
from tests.test_gpu_tokens import SHAPES


def case(lens, news, H, group, D, seed=1):
    r = np.random.default_rng(seed)
    for n, m in zip(lens, news):
        if m == 0:
            continue
        k = r.normal(size=(n, H, D)) * np.linspace(0.4, 1.2, n)[:, None, None]
        yield n, r.normal(size=(m, H * group, D)), k, r.normal(size=(n, H, D))


@pytest.mark.parametrize("lens,news,H,group,D,page", SHAPES + LONG)
def test_wrong_outputs_are_rejected(lens, news, H, group, D, page):
    if sum(n * m for n, m in zip(lens, news)) * H * group > 300000:
        lens, news = [n // 2 for n in lens], [max(1, min(m, 40)) for m in news]
    parts = {name: [] for name in ("right", "zeros", "left out", "equal")}
    for n, q, k, v in case(lens, news, H, group, D):
        out = tokens.attend(q, k, v, n)[0]
        parts["right"].append(out)
        parts["zeros"].append(np.zeros_like(out))
        there = np.ones(n, dtype=bool)
        there[n - n // 4:n - n // 8] = False
        parts["left out"].append(tokens.attend(q, k, v, n, exists=there)[0])
        first = np.arange(n) < n // 2
        a, b = (tokens.attend(q, k, v, n, exists=x)[0] for x in (first, ~first))
        parts["equal"].append(0.5 * (a + b) if n > 1 else a + b)
    parts = {name: np.concatenate(p) for name, p in parts.items()}
    right = parts["right"]
    rounded = torch.from_numpy(right).bfloat16().double().numpy()
    for dtype in ("bf16", "fp8"):
        # the limit of a q rotated in one term, the widest that the GPU's test uses
        limit = norm_limit(dtype, right.shape[0] * right.shape[1], 1.2)
        assert norm_error(rounded, right) <= limit
        assert norm_error(parts["zeros"], right) > limit
        if max(lens) > 1:
            assert norm_error(parts["left out"], right) > limit
            assert norm_error(parts["equal"], right) > limit


def test_non_finite_outputs_are_rejected():
    want = np.ones((2, 3))
    assert norm_error(np.full((2, 3), np.nan), want) == np.inf
    assert norm_error(want, np.zeros((2, 3))) == np.inf and norm_error(np.zeros(3), np.zeros(3)) == 0.0
