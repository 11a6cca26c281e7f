"""Heads turned by their position, and the cache write that turns its keys, on
the GPU against plain numpy forms in float64.

Tolerances (u = 2^-24): a head's norm is a sum of up to 16 squares a step and
6 levels, each rounded to float32, halved by the root, a division and two
products: under 14 u of each value.  Cosine and sine are off by the rest's own
rounding (2.5 u of at most pi / 4) and their sums' (2 u): 4 u, and the product
with amp: 5 u.  Two products and a sum: 2 u.  In all 21 u of amp (|a| + |b|),
and half a step of the output's type."""
import numpy as np
import pytest

from tests import q8_reference as R
from tests import rules_reference as X
from tests.gpu_util import announce
from tests.test_gpu_q8 import ROUND, U, Cache, _cu, _dev, _dtype, _np, _t, _typed

pytestmark = pytest.mark.gpu

TURN = 21 * U


def _freq(half, theta=10000.0):
    return (theta ** (-np.arange(half) / max(half, 1))).astype(np.float32)


def _near(got, want, size, dtype):
    rel, step = ROUND[dtype]
    err = np.abs(got.astype(np.float64) - want)
    return np.all(err <= (TURN * size) * (1 + rel) + rel * np.abs(want) + step + 1e-44)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 26), (128, 128), (128, 50), (128, 0), (256, 256),
                                     (80, 80), (96, 24), (2, 2), (10, 6), (512, 512), (130, 66),
                                     (64, 50), (64, 4), (64, 60), (512, 50), (100, 100)])
def test_turned_heads(dim, rot, interleaved, dtype):
    """Lengths from none to many, heads beside each other in one product's
    rows, with and without the norm, in place and not."""
    from bigvgan_waveform_decoder_amd import avae
    announce(f"qk_norm_rope dim {dim} rot {rot} interleaved {interleaved} {dtype}")
    rng = np.random.default_rng(dim * 1000 + rot)
    rope = avae.Rope(_dev(_freq(rot // 2)), interleaved, 1.25) if rot else None
    for heads, kv, new, lens in ((1, 1, [1], [1]), (6, 2, [1, 0, 5, 40], [2400, 7, 5, 100040]),
                                 (5, 0, [3], [900003]), (16, 3, [130], [131])):
        total = sum(new)
        qkv, f = _typed(rng.normal(size=(total, heads + 2 * kv, dim)) * np.exp(rng.normal(size=dim)),
                        dtype)
        w = [(1 + 0.3 * rng.normal(size=dim)).astype(np.float32) for _ in range(2)]
        pos = np.concatenate([np.arange(t - n, t) for n, t in zip(new, lens)])
        args = dict(cu=_dev(_cu(new)), lens=_dev(np.array(lens, np.int32)), max_rows=max(new))
        for norm in (False, True):
            qw, kw = (_dev(w[0]), _dev(w[1])) if norm else (None, None)
            want = [X.turn(f[:, lo:hi], pos, _freq(rot // 2), interleaved, 1.25,
                           g if norm else None)
                    for lo, hi, g in ((0, heads, w[0]), (heads, heads + kv, w[1]))]
            for inplace in (False, True):
                x = qkv.clone()
                q, k = x[:, :heads], x[:, heads:heads + kv] if kv else None
                gq, gk = avae.qk_norm_rope(q, k, rope, qw, kw, inplace=inplace, **args)
                assert _near(_np(gq), *want[0], dtype)
                if kv:
                    assert _near(_np(gk), *want[1], dtype)
                    rest = x[:, heads + kv:] if inplace else x
                    assert _t().equal(rest, qkv[:, heads + kv:] if inplace else qkv)
                else:
                    assert gk is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (128, 50, True), (96, 96, False)])
def test_turned_heads_at_odd_places(dim, rot, interleaved, dtype):
    """Heads that start at an odd element, a token's stride odd too, and a
    cache write of such keys."""
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    announce(f"qk_norm_rope at odd places dim {dim} rot {rot} {dtype}")
    rng = np.random.default_rng(dim)
    wide, f = _typed(rng.normal(size=(33, 3 * dim + 7)), dtype)
    x, xf = (t[:, 5:5 + 3 * dim].reshape(33, 3, dim) if isinstance(t, np.ndarray)
             else t[:, 5:5 + 3 * dim].unflatten(1, (3, dim)) for t in (wide, f))
    w = (1 + 0.3 * rng.normal(size=dim)).astype(np.float32)
    rope, args = avae.Rope(_dev(_freq(rot // 2)), interleaved), dict(cu=_dev(_cu([33])), lens=_dev(np.array([50], np.int32)))
    want = X.turn(xf, np.arange(17, 50), _freq(rot // 2), interleaved, 1.0, w)
    got, _ = avae.qk_norm_rope(x, None, rope, _dev(w), **args)
    assert _near(_np(got), *want, dtype)
    if dim in (64, 128):
        c = Cache(3, [50], 3, dim, 16)
        dev = c.upload()
        c.avae.kv_write_rope_q8(dev, x, x, _dev(c.table), args["cu"], args["lens"], rope, k_weight=_dev(w))
        _written(c, _cu([33]), None, *want, (c.k8.copy(), c.ks.copy()))
    # in place, what lies between stays
    before = wide.clone()
    avae.qk_norm_rope(x, None, rope, _dev(w), inplace=True, **args)
    assert _near(_np(x), *want, dtype)
    assert torch.equal(wide[:, :5], before[:, :5]) and torch.equal(wide[:, 5 + 3 * dim:], before[:, 5 + 3 * dim:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_turned_by_given_positions(dtype):
    """Positions beside, before and far after the rows' places; the same ones
    twice; with sequences and without."""
    from bigvgan_waveform_decoder_amd import avae
    announce(f"qk_norm_rope positions {dtype}")
    rng = np.random.default_rng(3)
    pos = np.array([0, 5, 5, -3, 2 ** 24 - 1, 70000, 1, 2, 0, 999999], np.int32)
    x, f = _typed(rng.normal(size=(10, 4, 128)), dtype)
    rope = avae.Rope(_dev(_freq(64)))
    want = X.turn(f, pos, _freq(64))
    for kw in ({}, dict(cu=_dev(_cu([4, 6])), lens=_dev(np.array([9, 6], np.int32)))):
        got, _ = avae.qk_norm_rope(x, None, rope, positions=_dev(pos), **kw)
        assert _near(_np(got), *want, dtype)
    # far beyond: the angle's own rounding in 64 bits, 2^-52 of it twice
    pos = np.array([2 ** 29 - 1, 2 ** 31 - 1, -2 ** 31] + 7 * [2 ** 28], np.int32)
    got, _ = avae.qk_norm_rope(x, None, rope, positions=_dev(pos))
    want, size = X.turn(f, pos, _freq(64))
    assert _near(_np(got), want, size * (1 + 2 ** 31 * 2.0 ** -51 / TURN), dtype)


def test_turned_rows_of_no_sequence_stay():
    """Rows behind the last sequence, rows between sequences that say they
    have none, offsets outside the rows; heads in the outer axis."""
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    announce("qk_norm_rope rows of no sequence")
    rng = np.random.default_rng(4)
    f = rng.normal(size=(12, 3, 64)).astype(np.float32)
    rope = avae.Rope(_dev(_freq(32)))
    for cu, mine in (([0, 5, 5, 9], range(9)), ([2, 6, 6, 8], range(2, 8)),
                     ([0, 4, 40, 2], range(4)), ([-3, 4, 9, 12], range(4, 12))):
        lens = np.array([8, 3, 4], np.int32)
        x = _dev(f.transpose(1, 0, 2)).transpose(0, 1)  # [tokens, heads] as [heads, tokens] in memory
        avae.qk_norm_rope(x, None, rope, cu=_dev(np.array(cu, np.int32)), lens=_dev(lens), inplace=True)
        pos = np.zeros(12)
        for b in range(3):
            n = cu[b + 1] - cu[b]
            if cu[b] >= 0 and 0 < n and cu[b + 1] <= 12:
                pos[cu[b]:cu[b + 1]] = np.arange(lens[b] - n, lens[b])
        want, size = X.turn(f, pos, _freq(32))
        mine = np.isin(np.arange(12), list(mine))
        assert _near(_np(x)[mine], want[mine], size[mine], "f32")
        assert np.array_equal(_np(x)[~mine], f[~mine])
    # a length below the rows' number: places before the first token
    x, f = _typed(f, "f32")
    got, _ = avae.qk_norm_rope(x, None, rope, cu=_dev(_cu([12])), lens=_dev(np.array([5], np.int32)))
    assert _near(_np(got), *X.turn(f, np.arange(-7, 5), _freq(32)), "f32")


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_head_norms_over_the_whole_range(eps):
    """Heads of zeros, of values whose squares leave float32 on either side,
    with an infinity and with a NaN; what is not turned is left alone."""
    from bigvgan_waveform_decoder_amd import avae
    announce(f"qk_norm_rope ranges eps {eps}")
    rng = np.random.default_rng(5)
    f = rng.normal(size=(1, 9, 128)).astype(np.float32)
    for h, by in enumerate((0.0, 1e-42, 1e-30, 1e-19, 1e-12, 1e18, 1e30, 1.0, 1.0)):
        f[0, h] *= np.float32(by)
    f[0, 7, 100], f[0, 8, 3] = np.inf, np.nan
    w = (1 + 0.3 * rng.normal(size=128)).astype(np.float32)
    rope = avae.Rope(_dev(_freq(16)))
    pos = np.array([77], np.int32)
    got = _np(avae.qk_norm_rope(_dev(f), None, rope, q_weight=_dev(w), eps=eps,
                                positions=_dev(pos))[0])
    want, size = X.turn(f, pos, _freq(16), weight=w, eps=np.float64(np.float32(eps)))
    assert (got[0, 0] == 0).all()
    assert _near(got[:, :7], want[:, :7], size[:, :7], "f32")
    assert np.isnan(got[0, 7, 100]) and (got[0, 7, :100] == 0).all() and np.isnan(got[0, 8]).all()
    # without a norm: an infinity beside turned dims, and in one pair
    x = np.ones((1, 1, 128), np.float32)
    x[0, 0, 40], x[0, 0, 3] = np.inf, np.inf
    got = _np(avae.qk_norm_rope(_dev(x), None, rope, positions=_dev(pos))[0])[0, 0]
    assert np.isposinf(got[40]) and not np.isfinite(got[[3, 19]]).any()
    assert np.isfinite(np.delete(got, [3, 19, 40])).all()


def test_turned_rows_past_one_launch():
    """More rows than the launch has waves: they are taken in turn."""
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    announce("qk_norm_rope 5 million rows")
    n = 5 * 2 ** 20 + 3
    x = torch.ones((n, 1, 2), device="cuda", dtype=torch.bfloat16)
    freq = torch.full((1,), 1e-3, device="cuda")
    got, _ = avae.qk_norm_rope(x, None, avae.Rope(freq), cu=_dev(_cu([n])),
                               lens=_dev(np.array([n], np.int32)))
    at = torch.arange(n, device="cuda", dtype=torch.float64) * freq.double()
    want = torch.stack((at.cos() - at.sin(), at.cos() + at.sin()), 1)
    assert float((got[:, 0].double() - want).abs().max()) <= 2.0 ** -8 * 1.5 + 1e-5


# ------------------------------------------------------------------ cache

def _written(c, cu, pos, keys, size, before):
    """Keys written at their places against float64 keys [tokens, heads, dim]."""
    k8, ks = _np(c.dev.k), _np(c.dev.k_scale)
    old8, olds = before
    for b, t in enumerate(c.lens):
        n = cu[b + 1] - cu[b]
        start = t - n
        for col in range(max(start, 0) // c.page, -(-t // c.page) if n > 0 else 0):
            p = c.table[b, col]
            lo, hi = max(start, col * c.page, 0), min(t, (col + 1) * c.page)
            rows = keys[cu[b] + lo - start:cu[b] + hi - start]
            err = TURN * size[cu[b] + lo - start:cu[b] + hi - start]
            held = lo - col * c.page
            for h in range(c.heads):
                top = np.abs(rows[:, h]).max()
                fresh = top / 127
                was = olds[p, h] if held else 0.0
                s = float(ks[p, h])
                near = err[:, h].max() / 127 + 2 * U * fresh
                assert s == was or abs(s - fresh) <= near
                assert abs(s - max(was, fresh)) <= near
                if s > was and held:
                    moved = R.quantise(old8[p, h, :held].astype(np.float32) * np.float32(was),
                                       np.float32(s))
                    assert np.array_equal(k8[p, h, :held], moved)
                else:
                    assert np.array_equal(k8[p, h, :held], old8[p, h, :held])
                off = np.abs(k8[p, h, held:hi - col * c.page] - rows[:, h] / s)
                assert np.all(off <= 0.5 + err[:, h] / s + 2.0 ** -16)
                old8[p, h, :hi - col * c.page] = k8[p, h, :hi - col * c.page]
                olds[p, h] = s
    assert np.array_equal(k8, old8) and np.array_equal(ks, olds, equal_nan=True)


WRITES = [  # new tokens, lengths afterwards, page
    ([1], [1], 16), ([1], [64], 64), ([1, 1, 1, 1], [17, 1, 32, 40], 16), ([0, 3, 0], [5, 3, 0], 32),
    ([5, 40, 100], [5, 90, 100], 64), ([300], [333], 128), ([16, 15, 17], [48, 31, 33], 16),
    ([1, 200, 7], [600, 256, 250], 256), ([4], [2], 16),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(WRITES)))
@pytest.mark.parametrize("heads,dim,rot,interleaved", [(1, 64, 64, True), (3, 128, 128, False),
                                                       (2, 256, 90, False), (2, 64, 30, True),
                                                       (2, 128, 64, False), (1, 64, 60, False),
                                                       (1, 64, 50, False), (2, 256, 4, False)])
def test_turned_cache_write(case, heads, dim, rot, interleaved, dtype):
    new, lens, page = WRITES[case]
    announce(f"kv_write_rope_q8 {new} {lens} page {page} heads {heads} dim {dim} rot {rot} {dtype}")
    rng = np.random.default_rng(case + 50)
    cu = _cu(new)
    total = cu[-1]
    spread = np.exp(1.5 * rng.normal(size=(total, heads, 1)))
    k, kf = _typed(rng.normal(size=(total, heads, dim)) * spread, dtype)
    v, vf = _typed(rng.normal(size=(total, heads, dim)), dtype)
    w = (1 + 0.3 * rng.normal(size=dim)).astype(np.float32)
    places = np.concatenate([np.arange(t - n, t) for n, t in zip(new, lens)])
    freq = _freq(rot // 2)
    for norm, given in ((False, False), (True, True)):
        c = Cache(case, lens, heads, dim, page)
        c.poison_unused()
        pos = rng.integers(0, 90000, size=total).astype(np.int32) if given else places
        want, size = X.turn(kf, pos, freq, interleaved, 1.25, w if norm else None)
        dev = c.upload()
        args = (_dev(c.table), _dev(cu), _dev(c.lens), c.avae.Rope(_dev(freq), interleaved, 1.25))
        kw = dict(k_weight=_dev(w) if norm else None, positions=_dev(pos) if given else None,
                  max_new=max(new))
        c.avae.kv_write_rope_q8(dev, k, v, *args, **kw)
        R.kv_write(c.v8, c.vs, vf, c.table, cu, lens, c.n, page)
        assert np.array_equal(_np(dev.v), c.v8)
        assert np.array_equal(_np(dev.v_scale), c.vs, equal_nan=True)
        _written(c, cu, pos, want, size, (c.k8.copy(), c.ks.copy()))
        # the same tokens again change nothing
        once = [t.clone() for t in (dev.k, dev.k_scale, dev.v)]
        c.avae.kv_write_rope_q8(dev, k, v, *args, **kw)
        for was, now in zip(once, (dev.k, dev.k_scale, dev.v)):
            assert np.array_equal(_np(was), _np(now), equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(WRITES)))
def test_untouched_keys_are_the_plain_writes(case, dtype):
    """Without norm and rotation, and at position 0 with neither angle nor
    gain, the plain write's bits."""
    new, lens, page = WRITES[case]
    announce(f"kv_write_rope_q8 as kv_write_q8 {new} {lens} {dtype}")
    rng = np.random.default_rng(case)
    cu = _cu(new)
    k, _ = _typed(rng.normal(size=(cu[-1], 2, 128)), dtype)
    v, _ = _typed(rng.normal(size=(cu[-1], 2, 128)), dtype)
    for how in range(3):
        c = Cache(case, lens, 2, 128, page)
        args = (_dev(c.table), _dev(cu), _dev(c.lens))
        one, two = c.upload(), c.upload()
        rope = None if how == 0 else c.avae.Rope(_dev(_freq(25 if how == 1 else 64)), how == 2)
        c.avae.kv_write_q8(one, k, v, *args)
        c.avae.kv_write_rope_q8(two, k, v, *args, rope,
                                positions=None if how == 0 else _dev(np.zeros(cu[-1], np.int32)))
        for a, b in ((one.k, two.k), (one.v, two.v), (one.k_scale, two.k_scale),
                     (one.v_scale, two.v_scale)):
            assert np.array_equal(_np(a), _np(b), equal_nan=True)


def test_turned_cache_write_bad_tables_and_values():
    """Table entries outside the cache leave their tokens out; a NaN key makes
    its page's scale NaN for its head and no other's; zeros stay zeros."""
    announce("kv_write_rope_q8 bad table and values")
    new, lens, page, heads, dim = [40, 20], [40, 70], 16, 2, 64
    c = Cache(5, lens, heads, dim, page)
    c.table[0, 1], c.table[0, 2] = c.n, -7
    c.table = np.ascontiguousarray(c.table[:, :4])
    cu = _cu(new)
    k = np.random.default_rng(3).normal(size=(60, heads, dim)).astype(np.float32)
    k[2, 1, 5] = np.nan
    k[40:, 0] = 0
    dev = c.upload()
    c.avae.kv_write_rope_q8(dev, _dev(k), _dev(k), _dev(c.table), _dev(cu), _dev(c.lens),
                            c.avae.Rope(_dev(_freq(32))), k_weight=_dev(np.ones(dim, np.float32)),
                            eps=0.0)
    ks, k8 = _np(dev.k_scale), _np(dev.k)
    untouched = [p for p in range(c.n) if p not in (c.table[0, 0], c.table[1, 3])]
    assert np.array_equal(k8[untouched], c.k8[untouched]) and np.array_equal(ks[untouched], c.ks[untouched])
    first, last = c.table[0, 0], c.table[1, 3]
    assert np.isnan(ks[first, 1]) and (k8[first, 1] == 0).all() and np.isfinite(ks[first, 0])
    assert ks[last, 0] == c.ks[last, 0] and (k8[last, 0, 2:] == 0).all()  # its first tokens are held
