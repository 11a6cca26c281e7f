"""Attention with rules where numbers leave float32 or its middle, in every
kernel (few rows, drafts, many rows) and type: scales of pages that are not
finite under a cap, factors past float32, caps far above and below the
scores, slopes as large as float32 holds."""
import numpy as np
import pytest

from tests import rules_reference as X
from tests.gpu_util import announce
from tests.test_gpu_attn_rules import _slopes
from tests.test_gpu_q8 import ROUND, U, Cache, _cu, _dev, _np, _typed

pytestmark = pytest.mark.gpu

# rows a cache head, two query heads each: 2 (few rows), 80 (drafts), 400 (many rows)
ROWS = [1, 40, 200]
TYPES = ["f32", "bf16", "f16"]


def _call(c, q, new, **kw):
    on = {k: _dev(v) if isinstance(v, np.ndarray) else v for k, v in kw.items()}
    out, lse = c.avae.attn_rules_q8(q, c.upload(), _dev(c.table), _dev(_cu(new)), _dev(c.lens),
                                    max_q=max(new), return_lse=True, **on)
    return _np(out), _np(lse)


# ------------------------------------------------------------------ what is not finite

@pytest.mark.parametrize("cap", [10.0, 300.0])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", ROWS)
def test_scales_that_are_not_finite_under_a_cap(rows, dtype, cap):
    """The rows that see such a page are NaN, in lse too, whatever the cap
    makes of an infinite score; the others as if it were not there."""
    announce(f"attn_rules_q8 scales not finite, {rows} rows, cap {cap} {dtype}")
    length = 500
    q, qf = _typed(np.random.default_rng(1).normal(size=(rows, 4, 64)), dtype)
    pos = np.arange(length - rows, length)
    key = np.arange(length)
    pre = np.array([50], np.int32)
    window = dict(window=40, prefix=pre, slopes=_slopes(4))
    for what, value in (("ks", np.nan), ("ks", np.inf), ("vs", np.nan), ("vs", np.inf)):
        for col, kw in ((1, window), ((length - 1) // 16, window), (7, {}), ((length - 1) // 16, {}),
                        ((length - rows // 2) // 16, {})):
            c = Cache(12, [length], 2, 64, 16)
            c.poison_unused()
            getattr(c, what)[c.table[0, col], 1] = value
            out, lse = _call(c, q, [rows], cap=cap, **kw)
            seen = key <= pos[:, None]
            if kw:
                seen = seen & (key > pos[:, None] - 40) | (key < 50)
            see = seen[:, 16 * col:16 * col + 16].any(1)
            want = np.repeat(see[:, None], 4, 1) & (np.arange(4) >= 2)
            assert np.array_equal(np.isnan(out).all(2), want)
            assert np.array_equal(np.isnan(out).any(2), want)
            assert np.array_equal(np.isnan(lse), want)
            getattr(c, what)[c.table[0, col], 1] = 0.01
            ref, rlse, weight, _, _ = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, _cu([rows]), [length],
                                                  16, 0.125, cap=cap, **kw)
            # (what the page's value is instead is in the reference of no row compared)
            assert np.all(np.abs(out - ref)[~want] <= (2.0 ** -9 if dtype == "bf16" else 2.0 ** -10) * weight[~want]
                          + ROUND[dtype][0] * np.abs(ref[~want]) + 1e-30)
            assert np.all(np.abs(lse - rlse)[~want] <= 1e-3)


# ------------------------------------------------------------------ caps

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", ROWS)
def test_factors_past_float32_with_large_scales(rows, dtype):
    """Key scales over 0.35 and quotients scale * |q| / cap past float32: a key
    that the query has nothing in common with scores 0, no NaN.  All scores
    lie within 1e-30 of each other, so the output is the values' mean: off by
    the probabilities' rounding (2^-11 in bfloat16, 2^-21 in the others'
    parts), by float32 sums of 300 terms in parts of 8 and the weights' 64
    roundings, and by its own."""
    announce(f"attn_rules_q8 large scales under a small cap, {rows} rows {dtype}")
    length = 300
    c = Cache(66, [length], 2, 64, 16)
    c.k8[:, :, ::3] = 0
    c.ks[:] = np.random.default_rng(3).uniform(0.36, 3.0, size=c.ks.shape)
    q = np.random.default_rng(1).normal(size=(rows, 4, 64))
    q = q / np.abs(q).max(2, keepdims=True)
    for scale, cap, gain in ((1e30, 1e-30, 60000.0), (-1e30, 1e-30, 33000.0), (3e38, 1e-30, 50000.0),
                             (1e38, 0.5, 60000.0)):
        dq, qf = _typed(q * gain, dtype)
        out, lse = _call(c, dq, [rows], scale=scale, cap=cap)
        if cap < 1e-3:
            ref, rlse, weight, _, _ = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, _cu([rows]), [length], 16,
                                                  scale, cap=cap)
            tol = (2 * (length / 8 + 64) * U + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21)) * weight
            assert np.all(np.abs(out - ref) <= tol + ROUND[dtype][0] * np.abs(ref) + ROUND[dtype][1])
            assert np.all(np.abs(lse - rlse) <= (length / 8 + 64) * U + 8 * U * np.abs(rlse))
        assert np.isfinite(out).all() and np.isfinite(lse).all()


@pytest.mark.parametrize("cap", [256.0, 257.0, 1e4, 1e6, 1e8, 1e30])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", ROWS)
def test_caps_far_above_the_scores(rows, dtype, cap):
    """A cap that no score comes near changes none.  A score's error: its
    float32 sum (dim + 24 roundings, query rows of float32 in 22 bits), the
    cap's: of 16-bit types up to 256 8 u cap (as in the tests of caps there),
    beyond and in float32 relative to the score, which is at most `size`: 2 for
    the factor, 2 for the series, 16 where (1 - e) / (1 + e) takes over at 0.25
    (the difference is off by 4 u of 0.24).  The factor over the cap may fall
    below float32's normal numbers: 2^-149 of it times a product of at most
    2^15 * 127 * dim, twice."""
    announce(f"attn_rules_q8 cap {cap}, {rows} rows {dtype}")
    length = 333
    c = Cache(70, [length], 2, 64, 32)
    c.poison_unused()
    for gain in (0.3, 2.0, 8.0):
        q, qf = _typed(np.random.default_rng(5).normal(size=(rows, 4, 64)) * gain, dtype)
        out, lse = _call(c, q, [rows], cap=cap)
        cap32 = float(np.float32(cap))
        ref, rlse, weight, size, _ = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, _cu([rows]), [length], 32,
                                                 0.125, cap=cap32)
        ds = (64 + 24 + 20) * U * size + (2.0 ** -21 * size if dtype == "f32" else 0)
        ds = ds + (8 * U * cap if dtype != "f32" and cap <= 256 else cap * 2.0 ** -148 * 2 ** 15 * 127 * 64)
        dp = 2 * np.expm1(ds) + (length / 8 + 64) * U + (2.0 ** -21 if dtype == "f32" else 2.0 ** -11)
        tol = dp[:, :, None] * weight + ROUND[dtype][0] * np.abs(ref) + ROUND[dtype][1]
        # (values below 2^-40 of the largest may count as 0)
        tol = tol + 2.0 ** -40 * 127 * length * np.nanmax(c.vs) + 1e-30
        assert ds.max() < 0.05  # the tolerance says something
        assert np.all(np.abs(out - ref) <= tol)
        assert np.all(np.abs(lse - rlse) <= ds + (length / 8 + 64) * U + 8 * U * np.abs(rlse))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", ROWS)
def test_caps_far_below_the_scores(rows, dtype):
    """Every score is the cap or its negative but for what tanh leaves: with
    caps of 1e-30 and 1e-3 at most 2 caps apart, so the scores' error is at
    most 8 u cap and the rest is the probabilities' and the sums'."""
    announce(f"attn_rules_q8 small caps, {rows} rows {dtype}")
    length = 333
    c = Cache(71, [length], 2, 64, 32)
    c.poison_unused()
    q, qf = _typed(np.random.default_rng(5).normal(size=(rows, 4, 64)) * 4, dtype)
    for cap in (1e-30, 1e-3):
        out, lse = _call(c, q, [rows], cap=cap)
        ref, rlse, weight, size, _ = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, _cu([rows]), [length], 32,
                                                 0.125, cap=float(np.float32(cap)))
        # a score's own error moves the capped one by at most as much, and by 2 caps
        ds = np.minimum((64 + 24) * U * size + (2.0 ** -21 * size if dtype == "f32" else 0), 2 * cap) + 8 * U * cap
        dp = 2 * np.expm1(ds) + (length / 8 + 64) * U + (2.0 ** -21 if dtype == "f32" else 2.0 ** -11)
        tol = dp[:, :, None] * weight + ROUND[dtype][0] * np.abs(ref) + ROUND[dtype][1] + 1e-30
        assert np.all(np.abs(out - ref) <= tol + 2.0 ** -40 * 127 * length * np.nanmax(c.vs))
        assert np.all(np.abs(lse - rlse) <= ds + (length / 8 + 64) * U + 8 * U * np.abs(rlse))


# ------------------------------------------------------------------ slopes

@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", ROWS)
def test_slopes_as_large_as_float32_holds(rows, dtype, cap):
    """Slopes are finite, of either sign: the nearest key alone is left, or
    the farthest, and nothing becomes NaN where slope * log2 e or the product
    with the distance passes float32.  The output is one value row: 8 bits
    times a scale, off by the weight's rounding and its own."""
    announce(f"attn_rules_q8 slopes at float32's end, {rows} rows {dtype}")
    length = 300
    c = Cache(72, [length], 2, 64, 16)
    c.poison_unused()
    q, qf = _typed(np.random.default_rng(5).normal(size=(rows, 4, 64)), dtype)
    slopes = np.array([3.4e38, -3.4e38, 1e30, -1e37], np.float32)
    out, lse = _call(c, q, [rows], slopes=slopes, cap=cap)
    v = (c.v8.astype(np.float64) * c.vs[:, :, None, None])[c.table[0]].transpose(1, 0, 2, 3).reshape(2, -1, 64)
    ref, rlse, _, size, _ = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, _cu([rows]), [length], 16, 0.125,
                                        cap=cap, slopes=slopes)
    pos = np.arange(length - rows, length)
    for h, at in ((0, pos), (1, 0 * pos), (2, pos), (3, 0 * pos)):
        want = v[h // 2][at]
        part = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
        tol = (part + 64 * U + ROUND[dtype][0]) * np.abs(want) + ROUND[dtype][1]
        tol = tol + 2.0 ** -40 * 127 * np.nanmax(c.vs) * length
        assert np.all(np.abs(out[:, h] - want) <= tol), h
        assert np.isfinite(lse[:, h]).all()
        if h in (0, 2):  # the key at the row itself: its score
            near = (64 + 24) * U * size[:, h] + (2.0 ** -21 * size[:, h] if dtype == "f32" else 0) + 8 * U * cap
            assert np.all(np.abs(lse[:, h] - rlse[:, h]) <= near + 64 * U + 8 * U * np.abs(rlse[:, h]))
    slopes[1] = np.nan
    out, lse = _call(c, q, [rows], slopes=slopes, cap=cap)
    assert np.array_equal(np.isnan(out).all((0, 2)), [False, True, False, False])
    assert np.array_equal(np.isnan(lse).any(0), [False, True, False, False])
