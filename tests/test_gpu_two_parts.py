"""Attention over the 8-bit cache, float32 outputs: the two float16 parts of a
probability are parts of one number."""
import numpy as np
import pytest

from tests import rules_reference as X
from tests.gpu_util import announce
from tests.test_gpu_q8 import U, Cache, _cu, _dev, _np, _typed

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["plain", "capped"])
@pytest.mark.parametrize("seqs,rows,length", [(1024, 1, 16), (400, 2, 40)])
def test_both_parts_are_of_the_same_product(seqs, rows, length, kind):
    """A probability times its value scale is rounded to float32 and then split.
    Where one part were taken from the unrounded product, the two would
    disagree by 2^-11 of the probability once in 2^14 keys (a tie of float16
    that the first rounding makes); here are over 2^17.  Scores are small, so
    that their own error (dim + 24 roundings of the products' sum, 2^-21 of
    them for the query's 22 bits) stays under a hundredth of that; the
    probabilities' is 2^-21 and the sums' len / 8 + 64 roundings, as in the
    other tests."""
    announce(f"two parts {kind} {seqs} x {rows} rows, {length} keys")
    c = Cache(91, [length] * seqs, 1, 64, 16)
    heads, new = 8, [rows] * seqs
    q, qf = _typed(np.random.default_rng(2).normal(size=(seqs * rows, heads, 64)) * 0.01, "f32")
    args = (q, c.upload(), _dev(c.table), _dev(_cu(new)), _dev(c.lens))
    kw = dict(cap=20.0) if kind == "capped" else {}
    out = c.avae.attn_rules_q8(*args, max_q=rows, **kw) if kw else c.avae.attn_q8(*args, max_q=rows)
    ref, _, weight, size, _ = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, _cu(new), list(c.lens), 16,
                                          0.125, **kw)
    ds = (64 + 24) * U * size + 2.0 ** -21 * size + 8 * U * min(kw.get("cap", 0.0), size.max())
    tol = (2 * np.expm1(ds) + (length / 8 + 64) * U + 2.0 ** -21)[:, :, None] * weight + U * np.abs(ref)
    assert tol.max() < 2.0 ** -11 / length * 127 * c.vs.max()  # one key's disagreement is over it
    assert np.all(np.abs(_np(out) - ref) <= tol), np.max(np.abs(_np(out) - ref) / tol)
