"""What an output of attention over a paged pool has to satisfy as a whole.

An elementwise bound has to allow the worst of every rounding at once, so over long
ranges it is wider than the output itself. Roundings are independent, though: their
2-norm is that of their root mean squares. A value rounded to bf16 is off by 2^-8 /
sqrt(3) of its binade's base at the root mean square, which over a binade's values is R =
1.7e-3 of the value; to fp16, R / 8. Relative to the 2-norm of an output whose V has
mean zero (so the output shrinks with the number of keys as the errors do):
  * the output's own rounding: R;
  * the weights': R over a bf16 pool, R / 8 over an 8-bit one;
  * a rotated q's, where it is kept in one term: R (R / 8) times the scores' standard deviation.
The limit is 1.35 times the root of the squares' sum. An output of few rows and heads
averages over few weights that stand for most of the mass: 1 + 2 / sqrt(rows x heads).
"""
import numpy as np

R = 1.7e-3


def norm_limit(dtype, rows_heads, score_std=0.0):
    """score_std: 0 where q is not rotated, or kept in two terms."""
    w = 1.0 if dtype == "bf16" else 1 / 64
    return 1.35 * R * np.sqrt(1 + w + w * score_std**2) * (1 + 2 / np.sqrt(rows_heads))


def norm_error(got, want):
    """|got - want| / |want| (0 for two zeros); NaN and infinities count as wrong."""
    if not np.all(np.isfinite(got)):
        return np.inf
    n = np.linalg.norm(want)
    return float(np.linalg.norm(got - want) / n) if n > 0 else (0.0 if not got.any() else np.inf)
