"""Attention with rules over the 8-bit cache (caps, biases by distance,
prefixes, trees of drafts) on the GPU against a plain numpy form in float64.

Tolerances: those of the attention without rules (a score's float32 sum and
the probabilities' rounding), and u = 2^-24 times
  8 cap: exp to 1.5 u, its sum, difference and reciprocal, and the product
    with the cap, none over 1;
  4 slope |p - t| a key: the slope in units of log2 e, its product and sum."""
import numpy as np
import pytest

from tests import q8_reference as R
from tests import rules_reference as X
from tests.gpu_util import announce
from tests.test_gpu_q8 import ROUND, U, Cache, _cu, _dev, _np, _t, _typed

pytestmark = pytest.mark.gpu


def _check(c, new, heads, dtype, seed, q=None, slack=0, max_len=None, gain=2.0, lines=None,
           tree=None, max_prefix=None, **rules):
    """One call with these rules against the plain form; returns the outputs."""
    rng = np.random.default_rng(seed)
    cu = _cu(new)
    if q is None:
        q = rng.normal(size=(cu[-1], heads, c.dim)) * gain
    dq, qf = _typed(q, dtype)
    args = (dq, c.upload(), _dev(c.table), _dev(cu), _dev(c.lens))
    on = {k: _dev(v) if isinstance(v, np.ndarray) else v for k, v in rules.items()}
    if lines is None:
        out, lse = c.avae.attn_rules_q8(*args, max_q=max(new) + slack, max_len=max_len,
                                        max_prefix=max_prefix, return_lse=True, **on)
    else:
        words = -(-(max(new) + slack) // 32)
        tree = _dev(X.tree_words(lines, words)) if tree is None else tree
        out, lse = c.avae.attn_tree_q8(*args, tree, max_q=max(new) + slack, max_len=max_len,
                                       return_lse=True, **on)
    rules.setdefault("scale", c.dim ** -0.5)
    ref, rlse, weight, size, bent = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, cu,
                                                list(c.lens), c.page, lines=lines, **rules)
    got, glse = _np(out), _np(lse)
    mine = np.zeros(cu[-1], bool)
    for b in range(len(new)):
        mine[cu[b]:cu[b + 1]] = True
    empty = np.isneginf(rlse)
    assert np.array_equal(np.isneginf(glse), empty)
    assert (got[empty] == 0).all()
    bad = np.isnan(rlse)
    assert np.array_equal(np.isnan(glse), bad)
    length = max(c.lens)
    cap = rules.get("cap", 0.0)
    ds = (c.dim + 24) * U * size + (2.0 ** -21 * size if dtype == "f32" else 0) + 8 * U * cap
    part = 2.0 ** -21 if dtype == "f32" else 2.0 ** -11
    with np.errstate(over="ignore"):
        dp = 2 * np.expm1(ds) + (length / 8 + 64) * U + part
    rel, step = ROUND[dtype]
    seen = c.table[(c.table >= 0) & (c.table < c.n)]
    step += 2.0 ** -40 * 127 * length * np.nanmax(c.vs[seen]) if seen.size else 0
    with np.errstate(invalid="ignore"):
        tol = dp[:, :, None] * weight + 4 * U * bent + rel * np.abs(ref) + step + 1e-30
        ok = np.abs(got - ref) <= tol
    ok |= np.isnan(ref) & np.isnan(got)
    assert ok.all(), (np.nanmax(np.abs(got - ref) / tol), np.argwhere(~ok)[:4])
    good = ~empty & ~bad
    reach = 0.0
    if rules.get("slopes") is not None:
        reach = 4 * U * np.abs(rules["slopes"]).max() * length
    near = ds + reach + (length / 8 + 64) * U + 8 * U * np.abs(np.where(good, rlse, 0))
    assert np.all(np.abs(glse[good] - rlse[good]) <= near[good])
    return out, lse


def _same_rows(a, b, c, qf, new, dtype, **rules):
    """Outputs of the kernels with rules and without.  With rules a score is
    rounded once more before its exponential (u of it, at most `size`), and
    the probabilities and sums are formed in another order (8 roundings): each
    probability is off by that twice, the output by so much of `weight`, and
    by two roundings to its type (float16 and bfloat16 probabilities are
    rounded to 2^-22 and 2^-11 on either side)."""
    _, _, weight, size, _ = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, _cu(new), list(c.lens),
                                        c.page, c.dim ** -0.5, **rules)
    part = {"f32": 2.0 ** -22, "f16": 2.0 ** -22, "bf16": 2.0 ** -11}[dtype]
    tol = (2 * U * (size + 8)[:, :, None] + 2 * part) * weight + 2 * ROUND[dtype][0] * np.abs(_np(b))
    ok = np.abs(_np(a) - _np(b)) <= tol + 2 * ROUND[dtype][1]
    return bool(ok.all())


def _slopes(heads, seed=0):
    s = 2.0 ** (-8 * np.arange(1, heads + 1) / heads)
    s[::3] *= -0.01  # of either sign
    return s.astype(np.float32)


ATTEND = [  # new, lengths, page
    ([1], [1], 16), ([1, 1, 1], [33, 16, 500], 16), ([1], [4099], 64),
    ([1, 0, 1, 1], [0, 7, 31, 257], 32), ([3, 1, 17], [3, 90, 140], 128), ([70], [70], 16),
    ([33, 65], [333, 65], 64), ([130], [1000], 256), ([5], [3], 16),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 64), (6, 2, 128), (3, 1, 256), (16, 1, 64)])
def test_caps_and_slopes(case, heads, kv_heads, dim, dtype):
    new, lens, page = ATTEND[case]
    announce(f"attn_rules_q8 cap, slopes {new} {lens} page {page} {heads}/{kv_heads} dim {dim} {dtype}")
    c = Cache(case + 10, lens, kv_heads, dim, page)
    c.poison_unused()
    _check(c, new, heads, dtype, case, cap=20.0)
    _check(c, new, heads, dtype, case, slopes=_slopes(heads))
    _check(c, new, heads, dtype, case, cap=3.0, slopes=_slopes(heads), gain=8.0, causal=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens,heads,kv_heads,dim,page", [
    ([1, 1], [700, 300], 4, 2, 64, 16), ([1], [5000], 6, 2, 128, 64), ([40, 90, 3], [300, 90, 3], 4, 2, 64, 32),
    ([200], [1300], 2, 2, 128, 128), ([17, 1], [40, 2000], 3, 1, 256, 16)])
@pytest.mark.parametrize("window", [0, 1, 33, 100, 900])
def test_prefixes(window, new, lens, heads, kv_heads, dim, page, dtype):
    """Prefixes from none past the length, with windows: what lies between is
    hidden, whatever its pages hold."""
    announce(f"attn_rules_q8 prefix window {window} {new} {lens} {heads}/{kv_heads} dim {dim} {dtype}")
    c = Cache(3, lens, kv_heads, dim, page)
    c.poison_unused()
    for i, p in enumerate((0, 1, 31, 64, 150, 10000)):
        prefix = np.array([max(p - 7 * b, 0) for b in range(len(new))], np.int32)
        first = np.array([(29 * b + 40) % 90 for b in range(len(new))], np.int32) if i % 2 else None
        d = Cache(3, lens, kv_heads, dim, page)
        d.poison_unused()
        # pages that no row sees may hold anything
        for b, (n, t) in enumerate(zip(new, lens)):
            lo = max(t - n - window + 1, 0) if window else 0
            for col in range(-(-t // page)):
                if col * page >= min(prefix[b], t) and (col + 1) * page <= lo:
                    d.ks[d.table[b, col]] = d.vs[d.table[b, col]] = np.nan
        _check(d, new, heads, dtype, i, window=window, prefix=prefix, first=first)
        _check(d, new, heads, dtype, i, window=window, prefix=prefix, first=first, cap=15.0,
               slopes=_slopes(heads), max_prefix=int(prefix.max()))


def test_a_prefix_longer_than_its_bound_is_cut():
    announce("attn_rules_q8 prefix past max_prefix")
    lens, new = [900, 500], [1, 1]
    c = Cache(4, lens, 2, 64, 16)
    args = (_dev(np.random.default_rng(1).normal(size=(2, 4, 64)).astype(np.float32)), c.upload(),
            _dev(c.table), _dev(_cu(new)), _dev(c.lens))
    long, cut = (_dev(np.array(p, np.int32)) for p in ([400, 90], [100, 90]))
    for window in (0, 50):
        a = c.avae.attn_rules_q8(*args, max_q=1, window=window, prefix=long, max_prefix=100)
        b = c.avae.attn_rules_q8(*args, max_q=1, window=window, prefix=cut, max_prefix=100)
        assert np.array_equal(_np(a), _np(b))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("new,lens,dim", [([1], [900], 64), ([2, 1], [300, 77], 128), ([64], [200], 128),
                                          ([50], [70], 256)])
def test_no_rule_is_the_plain_attention(new, lens, dim, dtype):
    """Nothing asked for: what attn_q8 gives."""
    announce(f"attn_rules_q8 without rules {new} {lens} dim {dim} {dtype}")
    c = Cache(8, lens, 2, dim, 16)
    _check(c, new, 4, dtype, 3)
    q, qf = _typed(np.random.default_rng(3).normal(size=(sum(new), 4, dim)), dtype)
    args = (q, c.upload(), _dev(c.table), _dev(_cu(new)), _dev(c.lens))
    a, b = c.avae.attn_rules_q8(*args, max_q=max(new)), c.avae.attn_q8(*args, max_q=max(new))
    assert _same_rows(a, b, c, qf, new, dtype)


def test_extreme_caps_and_queries():
    """Caps far below and above the scores, queries near both ends of float32:
    scores beyond a cap stand at it."""
    announce("attn_rules_q8 extremes")
    for new, lens in (([1], [300]), ([80], [200])):
        c = Cache(9, lens, 2, 64, 16)
        for cap in (1e-30, 1e-3, 1e4, 1e30):
            _check(c, new, 4, "f32", 5, cap=cap)
        q = np.random.default_rng(6).normal(size=(sum(new), 4, 64))
        _check(c, new, 4, "f32", 5, q=q * 2.0 ** -100, cap=10.0)
        for power in (60, 118):  # every score is the cap or its negative: the probabilities are exact
            out, _ = _check(c, new, 4, "f32", 5, q=q * 2.0 ** power, cap=10.0)
            qf = (q * 2.0 ** power).astype(np.float32)
            ref, _, weight, _, _ = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, _cu(new), lens, 16,
                                               0.125, cap=10.0)
            assert np.all(np.abs(_np(out) - ref) <= (200 * U + 2.0 ** -21) * weight)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens", [([1], [3000]), ([6], [400]), ([90], [500])])
def test_nan_pages_stay_with_the_rows_that_see_them(new, lens, dtype):
    """A key scale that is NaN or infinite, and a NaN value scale, under a cap
    (which an infinite score would pass): the rows that see the page are NaN,
    the others as if it were not there."""
    announce(f"attn_rules_q8 NaN pages {new} {lens} {dtype}")
    cu = _cu(new)
    q, qf = _typed(np.random.default_rng(1).normal(size=(cu[-1], 4, 64)), dtype)
    for what, value in (("ks", np.nan), ("ks", np.inf), ("vs", np.nan)):
        for col in (1, (lens[0] - 1) // 16):  # in the prefix, and in the window
            c = Cache(12, lens, 2, 64, 16)
            c.poison_unused()
            getattr(c, what)[c.table[0, col], 1] = value
            rules = dict(window=40, cap=10.0, slopes=_slopes(4))
            pre = np.array([50], np.int32)
            out, lse = c.avae.attn_rules_q8(q, c.upload(), _dev(c.table), _dev(cu), _dev(c.lens),
                                            max_q=max(new), window=40, cap=10.0, return_lse=True,
                                            slopes=_dev(_slopes(4)), prefix=_dev(pre))
            pos = np.arange(lens[0] - new[0], lens[0])
            key = np.arange(16 * col, min(16 * col + 16, lens[0]))
            see = ((key < 50) | (key <= pos[:, None]) & (key > pos[:, None] - 40)).any(1)
            assert np.array_equal(np.isnan(_np(out)).all(2), np.repeat(see[:, None], 4, 1) & (np.arange(4) >= 2))
            assert np.array_equal(np.isnan(_np(out)).any(2), np.isnan(_np(lse)))
            getattr(c, what)[c.table[0, col], 1] = 0.01
            ref = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, cu, lens, 16, 0.125, prefix=pre,
                              **rules)[0]
            ok = ~np.isnan(_np(out))
            scale = np.abs(ref).max()
            assert np.all(np.abs(_np(out) - ref)[ok] <= (1e-4 if dtype == "f32" else 0.02) * scale)


# ------------------------------------------------------------------ trees

def _parents(rng, new, width=5):
    out = []
    for n in new:
        out += [int(rng.integers(max(-1, i - width), i)) if i else -1 for i in range(n)]
    return np.array(out, np.int32)


TREES = [  # new, lengths, page
    ([1], [1], 16), ([1], [700], 64), ([24], [2423], 64), ([7, 1, 13], [7, 90, 140], 16),
    ([64], [300], 32), ([0, 33, 5], [12, 60, 2000], 16), ([100, 31], [100, 1000], 128), ([5], [3], 16),
    ([200], [333], 64),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(TREES)))
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 64), (6, 2, 128), (3, 1, 256), (16, 1, 64)])
def test_trees(case, heads, kv_heads, dim, dtype):
    new, lens, page = TREES[case]
    announce(f"attn_tree_q8 {new} {lens} page {page} {heads}/{kv_heads} dim {dim} {dtype}")
    rng = np.random.default_rng(case)
    c = Cache(case + 30, lens, kv_heads, dim, page)
    c.poison_unused()
    lines = X.lineage(_parents(rng, new), _cu(new))
    _check(c, new, heads, dtype, case, lines=lines)
    # any mask, a row of no draft at all among them; a first key; a cap
    lines = [[j for j in range(max(new)) if rng.random() < 0.4] for _ in lines]
    if lines:
        lines[0] = []
    first = np.array([max(t - n - 20, 0) for n, t in zip(new, lens)], np.int32)
    _check(c, new, heads, dtype, case, lines=lines, first=first, cap=10.0, slack=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens", [([20], [500]), ([90], [300])])
def test_a_chain_is_causal_attention(new, lens, dtype):
    """Each draft after the one before: the plain attention's rows."""
    announce(f"attn_tree_q8 chain {new} {lens} {dtype}")
    c = Cache(40, lens, 2, 128, 16)
    q, qf = _typed(np.random.default_rng(3).normal(size=(sum(new), 4, 128)), dtype)
    cu, lens_ = _dev(_cu(new)), _dev(c.lens)
    mask, pos = c.avae.tree_mask(_dev(np.arange(-1, new[0] - 1, dtype=np.int32)), cu, lens_)
    assert np.array_equal(_np(pos), np.arange(lens[0] - new[0], lens[0]))
    args = (q, c.upload(), _dev(c.table), cu, lens_)
    a, b = c.avae.attn_tree_q8(*args, mask), c.avae.attn_q8(*args)
    assert _same_rows(a, b, c, qf, new, dtype)


def test_drafts_of_other_branches_may_hold_anything():
    """A page of drafts that some rows see and others do not: its NaN stays
    with those, and so does the range of its value scale."""
    announce("attn_tree_q8 pages of other branches")
    for dtype in ("f32", "bf16"):
        for heads in (2, 8):
            new, lens = [40], [72]  # places 32 .. 71: pages 2, 3 and half of 4
            c = Cache(41, lens, 2, 64, 16)
            lines = [[i] if i < 16 else ([] if i < 32 else [0, 1]) + [i] for i in range(40)]
            c.vs[c.table[0, 3]] = np.nan
            q, qf = _typed(np.random.default_rng(3).normal(size=(40, heads, 64)), dtype)
            out = _np(c.avae.attn_tree_q8(q, c.upload(), _dev(c.table), _dev(_cu(new)),
                                          _dev(c.lens), _dev(X.tree_words(lines, 2))))
            assert np.array_equal(np.isnan(out).all((1, 2)), (np.arange(40) >= 16) & (np.arange(40) < 32))
            c.vs[c.table[0, 3]] = 1e30
            keep = np.r_[0:16, 32:40]
            out = _np(c.avae.attn_tree_q8(q, c.upload(), _dev(c.table), _dev(_cu(new)),
                                          _dev(c.lens), _dev(X.tree_words(lines, 2))))[keep]
            ref = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, _cu(new), lens, 16, 0.125,
                              lines=lines)[0][keep]
            assert np.abs(out - ref).max() <= (1e-5 if dtype == "f32" else 0.01) * np.abs(ref).max()


@pytest.mark.parametrize("new,lens", [([1], [1]), ([5, 0, 33, 64], [5, 3, 40, 900]), ([700, 1], [700, 2]),
                                      ([4096], [5000]), ([6], [4])])
def test_masks_from_parents(new, lens):
    from bigvgan_waveform_decoder_amd import avae
    announce(f"tree_mask {new} {lens}")
    rng = np.random.default_rng(7)
    cu = _cu(new)
    for width in (1, 3, 10000):
        parents = _parents(rng, new, width)
        for i in rng.integers(0, len(parents), size=len(parents) // 10):
            parents[i] = rng.choice([-5, 1 << 30, i, -1 << 31])  # none
        mask, pos = avae.tree_mask(_dev(parents), _dev(cu), _dev(np.array(lens, np.int32)),
                                   max_rows=max(new))
        lines = X.lineage(parents, cu)
        assert np.array_equal(_np(mask), X.tree_words(lines, -(-max(new) // 32)))
        start = np.concatenate([np.full(n, t - n) for n, t in zip(new, lens)])
        assert np.array_equal(_np(pos), start + [len(x) - 1 for x in lines])


def test_masks_of_rows_of_no_sequence_stay():
    from bigvgan_waveform_decoder_amd import avae
    announce("tree_mask slack rows")
    L = avae.lib()
    mask = _t().full((9, 4), 77, dtype=_t().int32, device="cuda")
    pos = _t().full((9,), 77, dtype=_t().int32, device="cuda")
    cu, lens = _dev(np.array([1, 4, 7], np.int32)), _dev(np.array([10, 3], np.int32))
    parents = _dev(np.array([0, -1, 0, 0, -1, 0, 1, 5, 5], np.int32))
    rows = avae.avae_ragged(cu.data_ptr(), lens.data_ptr(), None, 0, 0, 2, 9, 3)
    import ctypes
    assert L.avae_tree_mask(parents.data_ptr(), ctypes.addressof(rows), 3, mask.data_ptr(), 4,
                            pos.data_ptr(), None) == 0
    _t().cuda.synchronize()
    m = _np(mask)
    assert (m[[0, 7, 8]] == 77).all() and (m[:, 3] == 77).all() and (m[1:7, 1:3] == 0).all()
    assert m[1:7, 0].tolist() == [1, 3, 5, 1, 3, 7]
    assert _np(pos).tolist() == [77, 7, 8, 8, 0, 1, 2, 77, 77]
