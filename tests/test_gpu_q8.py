"""The 8-bit serving operators on the GPU against plain numpy forms.

Stored 8-bit values and rounded sums have to be equal: they are defined by
single float32 operations.  Tolerances of the rest are bounds on float32
rounding, given where they are used (u = 2^-24 is float32's unit roundoff)."""
import numpy as np
import pytest

from tests import q8_reference as R
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# half a unit in the last place of an output, relative (2^-p for p significant
# bits); float16 also has a smallest step
ROUND = {"f32": (U, 0.0), "bf16": (2.0 ** -8, 0.0), "f16": (2.0 ** -11, 2.0 ** -25)}


def _t():
    import torch
    return torch


def _dtype(name):
    torch = _t()
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _dev(a):
    return _t().from_numpy(np.ascontiguousarray(a)).cuda()


def _typed(a, name):
    """`a` (float64) on the device in the named type, and what that holds in float32."""
    t = _t().from_numpy(np.ascontiguousarray(a)).to(_dtype(name))
    return t.cuda(), t.float().numpy()


def _np(t):
    return t.detach().float().cpu().numpy() if t.is_floating_point() else t.detach().cpu().numpy()


def _round(a32, name):
    """float32 values rounded to the named type."""
    return _t().from_numpy(np.ascontiguousarray(a32)).to(_dtype(name)).float().numpy()


# ------------------------------------------------------------------ rows

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,C", [(1, 1), (3, 7), (1, 64), (5, 255), (2, 256), (7, 1000), (1, 1536),
                                 (33, 1537), (4, 4096), (3, 8192), (2, 8200), (2, 16384),
                                 (2, 33001)])
def test_norm_rows(M, C, dtype):
    from bigvgan_waveform_decoder_amd import avae
    announce(f"rms_norm_q8 [{M}, {C}] {dtype}")
    rng = np.random.default_rng(M * 100003 + C)
    x, xf = _typed(rng.normal(size=(M, C)) * np.exp(rng.normal(size=C)), dtype)
    r, rf = _typed(rng.normal(size=(M, C)) * 2, dtype)
    w = (1 + 0.2 * rng.normal(size=C)).astype(np.float32)
    # C/256 terms a lane and a short tree, in float32; the rest is a few roundings
    tol = (C / 256 + 24) * U
    for res in (None, r):
        q, s, h = avae.rms_norm_q8(x, _dev(w), eps=1e-6, residual=res)
        rq, rs, rh = R.rows_q8(xf, w, None if res is None else rf)
        assert np.array_equal(_np(q), rq)
        assert np.all(np.abs(_np(s) - rs) <= tol * rs)
        if res is None:
            assert h is None
        else:
            assert np.array_equal(_np(h), _round(rh, dtype))
    q, s = avae.quant_q8(x)
    rq, rs, _ = R.rows_q8(xf)
    assert np.array_equal(_np(q), rq) and np.array_equal(_np(s), rs.astype(np.float32))
    for out in ("f32", "bf16", "f16"):
        y = avae.dequant_q8(q, s, dtype=_dtype(out))
        assert np.array_equal(_np(y), _round(rq.astype(np.float32) * rs.astype(np.float32)[:, None],
                                             out))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_rows_strided_and_misaligned(dtype):
    """Rows of wider tensors, starting at an odd element."""
    from bigvgan_waveform_decoder_amd import avae
    for M, C, at in ((9, 520, 3), (6, 1537, 1), (4, 96, 5), (5, 4100, 7)):
        announce(f"rms_norm_q8 strided [{M}, {C}] at {at} {dtype}")
        rng = np.random.default_rng(C)
        x, xf = _typed(rng.normal(size=(M, C + 11)), dtype)
        r, rf = _typed(rng.normal(size=(M, C + 8)), dtype)
        w = _dev(np.concatenate([np.zeros(at, np.float32),
                                 (1 + rng.normal(size=C)).astype(np.float32)]))
        q, s, h = avae.rms_norm_q8(x[:, at:at + C], w[at:], residual=r[:, :C])
        rq, rs, rh = R.rows_q8(xf[:, at:at + C], _np(w)[at:], rf[:, :C])
        assert np.array_equal(_np(q), rq) and np.array_equal(_np(h), _round(rh, dtype))
        assert np.all(np.abs(_np(s) - rs) <= (C / 256 + 24) * U * rs)
        wide = _t().zeros((M, C + 13), dtype=_t().int8, device="cuda")
        wide[:, at:at + C] = q
        y = avae.dequant_q8(wide[:, at:at + C], s, dtype=_dtype(dtype))
        assert np.array_equal(_np(y), _round(rq.astype(np.float32) * _np(s)[:, None], dtype))


@pytest.mark.parametrize("C", [5, 1536, 9000])
def test_norm_rows_zero_and_non_finite(C):
    """A row of zeros, one below float32's normal range, one at its top, one
    with an infinity, one with a NaN, one whose largest values are ties at
    half a step."""
    from bigvgan_waveform_decoder_amd import avae
    announce(f"rms_norm_q8 edge rows C={C}")
    rng = np.random.default_rng(1)
    x = rng.normal(size=(7, C)).astype(np.float32)
    x[0] = 0
    x[1] = 1e-44
    x[2] *= 1e37 / np.abs(x[2]).max()
    x[3, C // 2] = np.inf
    x[4, C - 1] = np.nan
    x[5] = rng.integers(-254, 255, size=C) * 0.5  # scale 1: every odd one is a tie
    x[5, 0] = 127
    x[6] *= 1e-39
    for call, weight in ((lambda t: avae.quant_q8(t), None),
                         (lambda t: avae.rms_norm_q8(t, _t().ones(C, device="cuda"))[:2],
                          np.ones(C, np.float32))):
        q, s = call(_dev(x))
        rq, rs, _ = R.rows_q8(x, weight)
        assert np.array_equal(_np(q), rq)
        got = _np(s)
        assert got[0] == 0 and np.isnan(got[3]) and np.isnan(got[4])
        keep = [0, 5] if weight is not None else [0, 1, 2, 5, 6]
        assert np.all(np.abs(got[keep] - rs[keep]) <= (C / 256 + 24) * U * np.abs(rs[keep]))


@pytest.mark.parametrize("C", [3, 64, 1537, 33001])
def test_rows_smallest_scales(C):
    """Scales of a few of float32's smallest steps, rounded by up to a third:
    values past 127 of them stay at 127."""
    from bigvgan_waveform_decoder_amd import avae
    announce(f"quant_q8 smallest scales C={C}")
    rng = np.random.default_rng(C)
    tops = np.array([1, 63, 64, 127, 128, 190, 191, 317, 1000, 20000])
    x = rng.integers(-tops[:, None], tops[:, None] + 1, size=(len(tops), C))
    x[:, 0], x[:, -1] = tops, -tops
    x = (x * 2.0 ** -149).astype(np.float32)
    assert np.array_equal(x.astype(np.float64)[:, 0], tops * 2.0 ** -149)
    rq, rs, _ = R.rows_q8(x)
    q, s = avae.quant_q8(_dev(x))
    assert np.array_equal(_np(s).astype(np.float64), rs) and np.array_equal(_np(q), rq)
    rq, _, _ = R.rows_q8(x, np.ones(C, np.float32))
    assert np.array_equal(_np(avae.rms_norm_q8(_dev(x), _t().ones(C, device="cuda"))[0]), rq)


@pytest.mark.parametrize("dim", [64, 256])
def test_cache_smallest_scales(dim):
    announce(f"kv_write_q8 smallest scales dim {dim}")
    new, lens, page, heads = [256, 9], [256, 40], 256, 2
    c = Cache(11, lens, heads, dim, page)
    c.ks[c.table[1, 0]] = c.vs[c.table[1, 0]] = 2.0 ** -149
    cu = _cu(new)
    rng = np.random.default_rng(dim)
    k, v = ((rng.integers(-top, top + 1, size=(cu[-1], heads, dim)) * 2.0 ** -149)
            .astype(np.float32) for top in (190, 315))
    dev = c.upload()
    c.avae.kv_write_q8(dev, _dev(k), _dev(v), _dev(c.table), _dev(cu), _dev(c.lens))
    R.kv_write(c.k8, c.ks, k, c.table, cu, lens, c.n, page)
    R.kv_write(c.v8, c.vs, v, c.table, cu, lens, c.n, page)
    assert c.same()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_are_torchs_own(dtype):
    """Values and scales are to the bit what the same steps written in torch
    give on the device, so rows may come from either."""
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    announce(f"quant_q8 against torch's steps {dtype}")
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn((20011, 257), device="cuda", generator=gen).to(_dtype(dtype))
    q, s = avae.quant_q8(x)
    scale = x.float().abs().amax(1) / 127
    assert torch.equal(s, scale)
    assert torch.equal(q.float(), (x.float() / scale[:, None]).round())


def test_rows_none():
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    x = torch.empty((0, 40), device="cuda")
    q, s, h = avae.rms_norm_q8(x, torch.ones(40, device="cuda"), residual=x)
    assert q.shape == (0, 40) and s.shape == (0,) and h.shape == (0, 40)
    assert avae.dequant_q8(*avae.quant_q8(x)).shape == (0, 40)


# ------------------------------------------------------------------ product

def _linear_tol(ref, raw, bias, dtype, act):
    """Roundings of the sum to float32, of two products and of the bias's
    addition; SiLU's slope is below 1.1 and its exponential's relative error
    grows with the argument."""
    rel, step = ROUND[dtype]
    before = 5 * U * (np.abs(raw) + (0 if bias is None else np.abs(bias)))
    if act == "silu":
        before = 1.1 * before + (8 + 4 * np.abs(raw)) * U * np.abs(ref)
    return before + rel * np.abs(ref) + step + 1e-38


LINEAR = [(1, 1, 1), (1, 48, 32), (2, 17, 33), (1, 4608, 1536), (1, 1000, 100), (3, 64, 64),
          (5, 129, 257), (16, 256, 512), (17, 96, 1024), (31, 1536, 6144), (37, 1537, 1040),
          (64, 64, 8192), (65, 200, 48), (100, 512, 1536), (128, 128, 128), (129, 255, 320),
          (256, 256, 256), (257, 513, 640), (300, 1536, 1536), (513, 384, 1552), (1000, 300, 77),
          (2048, 2048, 512), (1025, 6144, 128)]


@pytest.mark.parametrize("M,N,K", LINEAR)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_linear(M, N, K, dtype):
    from bigvgan_waveform_decoder_amd import avae
    announce(f"linear_q8 {M}x{N}x{K} {dtype}")
    rng = np.random.default_rng(M + 7 * N + 31 * K)
    a = rng.integers(-127, 128, size=(M, K)).astype(np.int8)
    w = rng.integers(-127, 128, size=(N, K)).astype(np.int8)
    sa = np.exp(0.3 * rng.normal(size=M)).astype(np.float32) * np.float32(0.01)
    sw = np.exp(0.3 * rng.normal(size=N)).astype(np.float32) * np.float32(0.01 / np.sqrt(K))
    bias = rng.normal(size=N).astype(np.float32) * np.float32(0.1)
    raw = R.linear_q8(a, sa, w, sw)
    da, dsa, dw, dsw, db = (_dev(v) for v in (a, sa, w, sw, bias))
    for b, act in ((None, "none"), (bias, "silu"), (bias, "none")):
        y = avae.linear_q8(da, dsa, dw, dsw, bias=None if b is None else db, act=act,
                           dtype=_dtype(dtype))
        ref = R.linear_q8(a, sa, w, sw, b, act)
        err = np.abs(_np(y) - ref)
        assert np.all(err <= _linear_tol(ref, raw, b, dtype, act)), err.max()


@pytest.mark.parametrize("M,N,K,at,pad", [(5, 130, 300, 1, 3), (1, 64, 256, 8, 8), (40, 70, 65, 0, 1),
                                          (300, 300, 160, 16, 16), (20, 1000, 1000, 0, 24),
                                          (260, 512, 1536, 3, 0), (8, 256, 1536, 0, 5)])
def test_linear_strided_and_misaligned(M, N, K, at, pad):
    from bigvgan_waveform_decoder_amd import avae
    announce(f"linear_q8 strided {M}x{N}x{K} at {at} pad {pad}")
    rng = np.random.default_rng(K)
    a = rng.integers(-127, 128, size=(M, at + K + pad)).astype(np.int8)
    w = rng.integers(-127, 128, size=(N, at + K + pad)).astype(np.int8)
    one_m, one_n = np.ones(M, np.float32), np.ones(N, np.float32)
    da, dw = _dev(a), _dev(w)
    y = avae.linear_q8(da[:, at:at + K], _dev(one_m), dw[:, at:at + K], _dev(one_n))
    ref = R.linear_q8(a[:, at:at + K], one_m, w[:, at:at + K], one_n)
    assert np.all(np.abs(_np(y) - ref) <= 2 * U * np.abs(ref))


def test_linear_extremes():
    """The largest sums that fit, scales of zero and NaN, and a long K."""
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    for M, N, K in ((2, 3, 131071), (70, 65, 100000), (300, 130, 40000)):
        announce(f"linear_q8 extremes {M}x{N}x{K}")
        a = np.full((M, K), -128, np.int8)
        w = np.full((N, K), -128, np.int8)
        w[1] = 127
        sa = np.ones(M, np.float32)
        sa[0], sa[1] = np.nan, 0
        y = _np(avae.linear_q8(_dev(a), _dev(sa), _dev(w), torch.ones(N, device="cuda")))
        ref = R.linear_q8(a, sa, w, np.ones(N, np.float32))
        assert np.isnan(y[0]).all() and (y[1] == 0).all()
        assert np.all(np.abs(y[2:] - ref[2:]) <= 2 * U * np.abs(ref[2:]))
    assert avae.linear_q8(torch.empty((0, 32), dtype=torch.int8, device="cuda"),
                          torch.empty(0, device="cuda"),
                          torch.zeros((5, 32), dtype=torch.int8, device="cuda"),
                          torch.ones(5, device="cuda")).shape == (0, 5)


# ------------------------------------------------------------------ cache

class Cache:
    """A cache with random contents, its page table, and host copies."""

    def __init__(self, seed, lens, heads, dim, page, spare=3):
        from bigvgan_waveform_decoder_amd import avae
        rng = np.random.default_rng(seed)
        pages = [-(-t // page) for t in lens]
        n = sum(pages) + spare
        order = rng.permutation(n)
        self.table = np.full((len(lens), max(pages + [1])), -1, np.int32)
        at = 0
        for b, c in enumerate(pages):
            self.table[b, :c] = order[at:at + c]
            at += c
        shape = (n, heads, page, dim)
        self.k8, self.v8 = (rng.integers(-127, 128, size=shape).astype(np.int8) for _ in range(2))
        self.ks, self.vs = (np.exp(rng.normal(size=(n, heads)) * 0.5).astype(np.float32)
                            * np.float32(0.015) for _ in range(2))
        self.spare = order[at:]
        self.lens = np.array(lens, np.int32)
        self.page, self.dim, self.heads, self.n = page, dim, heads, n
        self.avae = avae

    def poison_unused(self):
        """What no sequence may look at: scales of unused pages and heads."""
        self.ks[self.spare] = np.nan
        self.vs[self.spare] = np.nan

    def upload(self):
        self.dev = self.avae.KvCacheQ8(_dev(self.k8), _dev(self.v8), _dev(self.ks), _dev(self.vs))
        return self.dev

    def same(self):
        return (np.array_equal(_np(self.dev.k), self.k8) and np.array_equal(_np(self.dev.v), self.v8)
                and np.array_equal(_np(self.dev.k_scale), self.ks, equal_nan=True)
                and np.array_equal(_np(self.dev.v_scale), self.vs, equal_nan=True))


def _cu(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


WRITES = [  # new tokens, lengths afterwards, page
    ([1], [1], 16), ([1], [64], 64), ([1, 1, 1, 1], [17, 1, 32, 40], 16), ([0, 3, 0], [5, 3, 0], 32),
    ([5, 40, 100], [5, 90, 100], 64), ([300], [333], 128), ([16, 15, 17], [48, 31, 33], 16),
    ([1, 200, 7], [600, 256, 250], 256), ([4], [2], 16),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(WRITES)))
@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 128), (2, 256)])
def test_cache_write_and_read(case, dtype, heads, dim):
    new, lens, page = WRITES[case]
    announce(f"kv_write_q8 {new} {lens} page {page} heads {heads} dim {dim} {dtype}")
    c = Cache(case, lens, heads, dim, page)
    c.poison_unused()
    rng = np.random.default_rng(case + 50)
    cu = _cu(new)
    # ranges around the held ones: some pages grow, some keep their scale
    spread = np.exp(1.5 * rng.normal(size=(cu[-1], heads, 1)))
    k, kf = _typed(rng.normal(size=(cu[-1], heads, dim)) * spread, dtype)
    v, vf = _typed(rng.normal(size=(cu[-1], heads, dim)), dtype)
    dev = c.upload()
    args = (_dev(c.table), _dev(cu), _dev(c.lens))
    for again in range(2):  # the second time changes nothing
        c.avae.kv_write_q8(dev, k, v, *args, max_new=max(new))
        if not again:
            R.kv_write(c.k8, c.ks, kf, c.table, cu, lens, c.n, page)
            R.kv_write(c.v8, c.vs, vf, c.table, cu, lens, c.n, page)
        assert c.same()
    for out in ("f32", dtype):
        back = _cu([min(t, n + 5) for n, t in zip(new, lens)])
        rk, rv = c.avae.kv_read_q8(dev, args[0], _dev(back), args[2], total=int(back[-1]),
                                   dtype=_dtype(out))
        assert np.array_equal(_np(rk), _round(R.kv_read(c.k8, c.ks, c.table, back, lens, page), out))
        assert np.array_equal(_np(rv), _round(R.kv_read(c.v8, c.vs, c.table, back, lens, page), out))


def test_cache_write_strided_rows():
    """Keys and values as parts of one packed projection, heads not next to each other."""
    announce("kv_write_q8 strided")
    new, lens, page, heads, dim = [3, 20], [40, 20], 16, 2, 64
    c = Cache(3, lens, heads, dim, page)
    cu = _cu(new)
    rng = np.random.default_rng(9)
    for width, off in ((5 * heads * dim, 2 * dim), (5 * heads * dim + 1, 3)):
        packed, pf = _typed(rng.normal(size=(cu[-1], width)), "bf16")
        k = packed[:, off:off + 2 * heads * dim].unflatten(1, (heads, 2 * dim))[:, :, :dim]
        v = packed[:, off:off + 2 * heads * dim].unflatten(1, (heads, 2 * dim))[:, :, dim:]
        both = pf[:, off:off + 2 * heads * dim].reshape(cu[-1], heads, 2 * dim)
        dev = c.upload()
        c.avae.kv_write_q8(dev, k, v, _dev(c.table), _dev(cu), _dev(c.lens))
        R.kv_write(c.k8, c.ks, both[:, :, :dim], c.table, cu, lens, c.n, page)
        R.kv_write(c.v8, c.vs, both[:, :, dim:], c.table, cu, lens, c.n, page)
        assert c.same()


def test_cache_non_finite_and_zero():
    """A NaN or infinity poisons its page and head alone; zeros have scale 0;
    a page written from its start forgets what it was."""
    announce("kv_write_q8 non-finite")
    new, lens, page, heads, dim = [20, 4], [20, 36], 16, 2, 64
    c = Cache(4, lens, heads, dim, page)
    c.ks[c.table[0, 0]] = np.nan  # left over from an earlier use
    cu = _cu(new)
    rng = np.random.default_rng(2)
    k = rng.normal(size=(cu[-1], heads, dim)).astype(np.float32)
    v = rng.normal(size=(cu[-1], heads, dim)).astype(np.float32)
    k[3, 1, 5] = np.nan
    k[17, 0, 0] = -np.inf
    v[:16, 0] = 0
    v[22, 1, 63] = np.inf
    dev = c.upload()
    c.avae.kv_write_q8(dev, _dev(k), _dev(v), _dev(c.table), _dev(cu), _dev(c.lens))
    R.kv_write(c.k8, c.ks, k, c.table, cu, lens, c.n, page)
    R.kv_write(c.v8, c.vs, v, c.table, cu, lens, c.n, page)
    assert c.same()
    assert np.isnan(c.ks[c.table[0, 0], 1]) and np.isfinite(c.ks[c.table[0, 0], 0])
    assert c.vs[c.table[0, 0], 0] == 0


def test_cache_table_entries_that_are_no_page():
    """Table entries outside the cache, and lengths past the table: those
    tokens are left out, nothing else is touched."""
    announce("kv_write_q8 bad table")
    new, lens, page, heads, dim = [40, 20], [40, 70], 16, 1, 64
    c = Cache(5, lens, heads, dim, page)
    c.table[0, 1], c.table[0, 2] = c.n, -7
    c.table = np.ascontiguousarray(c.table[:, :4])  # 64 tokens: the second sequence has 70
    cu = _cu(new)
    rng = np.random.default_rng(3)
    k, v = (rng.normal(size=(cu[-1], heads, dim)).astype(np.float32) for _ in range(2))
    dev = c.upload()
    args = (_dev(c.table), _dev(cu), _dev(c.lens))
    c.avae.kv_write_q8(dev, _dev(k), _dev(v), *args)
    R.kv_write(c.k8, c.ks, k, c.table, cu, lens, c.n, page)
    R.kv_write(c.v8, c.vs, v, c.table, cu, lens, c.n, page)
    assert c.same()
    rk, rv = c.avae.kv_read_q8(dev, *args, total=int(cu[-1]))
    assert np.array_equal(_np(rk), R.kv_read(c.k8, c.ks, c.table, cu, lens, page))
    assert np.array_equal(_np(rv), R.kv_read(c.v8, c.vs, c.table, cu, lens, page))
    assert (_np(rk)[16:40] == 0).all()


# ------------------------------------------------------------------ attention

def _check_attention(c, new, heads, dtype, seed, causal=True, window=0, first=None, scale=None,
                     q=None, slack=0, max_len=None):
    rng = np.random.default_rng(seed)
    cu = _cu(new)
    if q is None:
        q = rng.normal(size=(cu[-1], heads, c.dim)) * 2
    dq, qf = _typed(q, dtype)
    sc = c.dim ** -0.5 if scale is None else scale
    out, lse = c.avae.attn_q8(dq, c.upload(), _dev(c.table), _dev(cu), _dev(c.lens),
                              max_q=max(new) + slack, max_len=max_len, scale=scale, causal=causal,
                              window=window, first=None if first is None else _dev(first),
                              return_lse=True)
    ref, rlse, weight, size = R.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, cu, list(c.lens),
                                          c.page, sc, causal, window, first)
    got, glse = _np(out), _np(lse)
    empty = np.isneginf(rlse)
    assert np.array_equal(np.isneginf(glse), empty)
    assert (got[empty] == 0).all()
    bad = np.isnan(rlse)
    assert np.array_equal(np.isnan(glse), bad)
    # Score: dim float32 additions, a few roundings, and for float32 queries
    # the 22 bits they are multiplied with; the products of one row sum to at
    # most `size`.  Probabilities: the score's error, their own rounding
    # (2^-11 in float16, 2^-22 in two parts), the sums over the keys.  float16
    # has a smallest step too: with the row's largest probability and value
    # scale at 2^15, half of it is 2^-40 of that scale for each key.
    length = max(c.lens)
    ds = (c.dim + 16) * U * size + (2.0 ** -21 * size if dtype == "f32" else 0)
    dp = 2 * np.expm1(ds) + (length / 8 + 64) * U + (2.0 ** -21 if dtype == "f32" else 2.0 ** -11)
    rel, step = ROUND[dtype]
    seen = c.table[(c.table >= 0) & (c.table < c.n)]
    step += 2.0 ** -40 * 127 * length * np.nanmax(c.vs[seen]) if seen.size else 0
    with np.errstate(invalid="ignore"):
        tol = dp[:, :, None] * weight + rel * np.abs(ref) + step + 1e-30
        ok = np.abs(got - ref) <= tol
    ok |= np.isnan(ref) & np.isnan(got)
    assert ok.all(), (np.nanmax(np.abs(got - ref) / tol), np.argwhere(~ok)[:4])
    good = ~empty & ~bad
    near = ds + (length / 8 + 64) * U + 8 * U * np.abs(np.where(good, rlse, 0))
    assert np.all(np.abs(glse[good] - rlse[good]) <= near[good])


ATTEND = [  # new, lengths, page
    ([1], [1], 16), ([1], [2], 64), ([1, 1, 1], [33, 16, 500], 16), ([1], [4099], 64),
    ([1, 0, 1, 1], [0, 7, 31, 257], 32), ([3, 1, 17], [3, 90, 140], 128), ([70], [70], 16),
    ([33, 65], [333, 65], 64), ([130], [1000], 256), ([5], [3], 16),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 64), (6, 2, 128), (4, 4, 128), (3, 1, 256),
                                                (16, 1, 64)])
def test_attention(case, heads, kv_heads, dim, dtype):
    new, lens, page = ATTEND[case]
    announce(f"attn_q8 {new} {lens} page {page} heads {heads}/{kv_heads} dim {dim} {dtype}")
    c = Cache(case + 10, lens, kv_heads, dim, page)
    c.poison_unused()
    _check_attention(c, new, heads, dtype, case)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,causal", [(1, True), (16, True), (100, True), (5000, True), (0, False)])
def test_attention_windows(window, causal, dtype):
    """Sliding windows around the tiles' sizes, and no order at all."""
    new, lens, page = [1, 40, 90], [700, 300, 90], 32
    announce(f"attn_q8 window {window} causal {causal} {dtype}")
    c = Cache(21, lens, 2, 64, page)
    c.poison_unused()
    _check_attention(c, new, 8, dtype, 5, causal=causal, window=window)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_first_key(causal):
    """Keys before a sequence's first are hidden: rows before it see nothing."""
    new, lens = [20, 1, 64, 1], [300, 77, 64, 50]
    announce(f"attn_q8 first causal {causal}")
    c = Cache(22, lens, 2, 128, 16)
    c.poison_unused()
    # the pages before the first key may hold anything
    for b, f in enumerate((290, 40, 30, 50)):
        for col in range(f // 16):
            c.ks[c.table[b, col]] = np.nan
            c.vs[c.table[b, col]] = np.nan
    for dtype in ("f32", "bf16"):
        _check_attention(c, new, 6, dtype, 6, causal=causal,
                         first=np.array([290, 40, 30, 50], np.int32))
        _check_attention(c, new, 6, dtype, 6, causal=causal, window=25 if causal else 0,
                         first=np.array([290, 40, 30, 500], np.int32))


def test_attention_poisoned_page_stays_with_the_rows_that_see_it():
    """A page whose scale is NaN makes the rows that see it NaN, no other."""
    new, lens = [48, 1], [80, 40]
    announce("attn_q8 NaN page")
    c = Cache(23, lens, 2, 64, 16)
    c.poison_unused()
    c.vs[c.table[0, 3], 0] = np.nan  # tokens 48..63 of the first sequence
    c.ks[c.table[0, 4], 1] = np.nan  # tokens 64..79
    for dtype in ("f32", "bf16"):
        rng = np.random.default_rng(7)
        q, qf = _typed(rng.normal(size=(49, 4, 64)), dtype)
        cu = _cu(new)
        out = _np(c.avae.attn_q8(q, c.upload(), _dev(c.table), _dev(cu), _dev(c.lens)))
        pos = np.arange(32, 80)
        assert np.array_equal(np.isnan(out[:48, :2]).any(2), np.repeat((pos >= 48)[:, None], 2, 1))
        assert np.array_equal(np.isnan(out[:48, 2:]).any(2), np.repeat((pos >= 64)[:, None], 2, 1))
        assert np.isfinite(out[48]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_ranges(dtype):
    """Large and small queries, scales far apart between pages, zero pages, a
    softmax that one key takes whole, and one that all share."""
    announce(f"attn_q8 ranges {dtype}")
    lens, new = [200, 200, 64, 130], [2, 2, 2, 2]
    c = Cache(24, lens, 2, 128, 16)
    c.poison_unused()
    rng = np.random.default_rng(8)
    for b in range(4):
        for col in range(-(-lens[b] // 16)):
            p = c.table[b, col]
            c.vs[p] *= np.float32(10.0 ** rng.integers(-6, 4))
            if col % 5 == 3:
                c.vs[p], c.v8[p] = 0, 0
    c.vs[c.table[2, :4]] = 0
    c.v8[c.table[2, :4]] = 0
    q = rng.normal(size=(8, 4, 128))
    q[0] *= 1e-30
    q[1] *= 30
    q[2] = 0
    q[3, :, 7] *= 200
    _check_attention(c, new, 4, dtype, 0, q=q)
    _check_attention(c, new, 4, dtype, 0, q=q * 1e-3, scale=3.0)
    _check_attention(c, new, 4, dtype, 0, q=q, scale=-0.05)


def test_attention_bad_table_and_slack():
    """Entries that are no page hide their tokens; larger bounds than needed
    for the rows and the length change nothing."""
    new, lens = [3, 1], [100, 60]
    announce("attn_q8 bad table")
    c = Cache(25, lens, 1, 64, 16)
    c.table[0, 2] = c.n + 5
    c.table[0, 5] = -1
    c.table[1, :] = -2
    for dtype in ("f32", "bf16"):
        _check_attention(c, new, 2, dtype, 1, slack=1)
        _check_attention(c, new, 2, dtype, 1, max_len=112)


def test_attention_strided_queries_and_another_stream():
    """Queries as part of a packed projection, the whole call on a side stream."""
    torch = _t()
    announce("attn_q8 strided, side stream")
    new, lens = [5, 1], [50, 300]
    c = Cache(26, lens, 2, 64, 32)
    cu = _cu(new)
    rng = np.random.default_rng(4)
    for off in (0, 64, 3):
        packed, pf = _typed(rng.normal(size=(6, 8 * 64 + 5)), "bf16")
        q = packed[:, off:off + 4 * 64].unflatten(1, (4, 64))
        dev = c.upload()
        args = (_dev(c.table), _dev(cu), _dev(c.lens))
        want = c.avae.attn_q8(q, dev, *args)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = c.avae.attn_q8(q, dev, *args)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        ref = R.attention(pf[:, off:off + 256].reshape(6, 4, 64), c.k8, c.ks, c.v8, c.vs, c.table,
                          cu, lens, 32, 0.125)[0]
        assert np.abs(_np(got) - ref).max() <= 0.02


def test_attention_reads_the_cache_in_any_page_order():
    """The same tokens in other pages give the same bits."""
    torch = _t()
    announce("attn_q8 page order")
    lens, new = [900, 130], [1, 30]
    a = Cache(27, lens, 2, 128, 16)
    b = Cache(28, lens, 2, 128, 16)
    for s in range(2):
        for col in range(-(-lens[s] // 16)):
            src, dst = a.table[s, col], b.table[s, col]
            b.k8[dst], b.v8[dst], b.ks[dst], b.vs[dst] = a.k8[src], a.v8[src], a.ks[src], a.vs[src]
    cu = _cu(new)
    q = torch.randn((31, 8, 128), device="cuda", generator=torch.Generator("cuda").manual_seed(1),
                    dtype=torch.float32).bfloat16()
    outs = [x.avae.attn_q8(q, x.upload(), _dev(x.table), _dev(cu), _dev(x.lens)) for x in (a, b)]
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens,heads,kv_heads,dim,page", [
    ([1, 1, 1], [3000, 1, 1777], 4, 2, 64, 16), ([1], [9001], 2, 1, 128, 64),
    ([4, 2], [5000, 130], 12, 4, 128, 32), ([1, 1], [2500, 2048], 3, 1, 256, 128)])
def test_attention_long(new, lens, heads, kv_heads, dim, page, dtype):
    """Few rows over many keys: the keys are split and joined."""
    announce(f"attn_q8 long {new} {lens} {heads}/{kv_heads} dim {dim} page {page} {dtype}")
    c = Cache(31, lens, kv_heads, dim, page)
    c.poison_unused()
    _check_attention(c, new, heads, dtype, 9)
    _check_attention(c, new, heads, dtype, 9, window=1000)
    _check_attention(c, new, heads, dtype, 9,
                     first=np.array([2000] * len(lens), np.int32))


def test_attention_pages_next_to_the_seen_keys_may_hold_anything():
    """Pages outside the window, in the same 32 keys as seen ones, with
    scales of NaN, infinity and the largest float32."""
    announce("attn_q8 neighbours")
    new, lens = [1, 1], [115, 400]
    for bad in (np.nan, np.inf, 3e38):
        c = Cache(32, lens, 1, 64, 16)
        c.poison_unused()
        for b, lo in ((0, 112), (1, 304)):  # windows of 3 and 96 keys
            for col in range(lo // 16):
                c.ks[c.table[b, col]] = bad
                c.vs[c.table[b, col]] = bad
        c.table = np.concatenate([c.table, np.full((2, 1), c.spare[0], np.int32)], 1)
        c.ks[c.spare[0]] = c.vs[c.spare[0]] = bad
        c.table[0, 8] = c.spare[0]  # past the first sequence's length
        for dtype in ("f32", "bf16"):
            _check_attention(c, new, 2, dtype, 3, first=np.array([112, 304], np.int32))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("new,lens,heads,kv_heads,dim,page,window", [
    ([200], [200], 1, 1, 64, 16, 0), ([129, 40], [700, 40], 3, 1, 128, 64, 0),
    ([300, 1, 0, 77], [300, 600, 0, 1100], 4, 2, 128, 32, 0), ([100], [1500], 8, 2, 64, 128, 0),
    ([64], [3000], 4, 2, 128, 16, 0), ([150], [900], 2, 1, 256, 16, 0), ([260], [1300], 2, 2, 64, 32, 70),
    ([33], [2000], 4, 1, 128, 256, 900), ([130], [100], 2, 2, 64, 16, 0)])
def test_attention_many_rows(new, lens, heads, kv_heads, dim, page, window, dtype):
    """Prompts and long drafts: rows over several workgroups, keys split and not."""
    announce(f"attn_q8 many {new} {lens} {heads}/{kv_heads} dim {dim} page {page} window {window} {dtype}")
    c = Cache(41, lens, kv_heads, dim, page)
    c.poison_unused()
    _check_attention(c, new, heads, dtype, 10, window=window)
    first = np.array([17 + 300 * (t > 1000) for t in lens], np.int32)
    _check_attention(c, new, heads, dtype, 11, window=window, first=first)
    if not window:
        _check_attention(c, new, heads, dtype, 12, causal=False, first=first)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_lengths_past_the_table(dtype):
    """A length beyond the table's tokens adds no key: few and many rows."""
    announce(f"attn_q8 lengths past the table {dtype}")
    for new in ([1, 2], [60, 3]):
        c = Cache(33, [64, 64], 2, 64, 16)
        c.poison_unused()
        c.table = np.ascontiguousarray(c.table[:, :4])
        c.lens = np.array([1000, 70], np.int32)
        _check_attention(c, new, 4, dtype, 2, max_len=64)


def test_cache_beyond_32_bit_offsets():
    """Pages whose first byte lies past 4 GiB of the cache."""
    announce("kv_write_q8, kv_read_q8, attn_q8 past 4 GiB")
    torch = _t()
    from bigvgan_waveform_decoder_amd import avae
    pages, page, dim = 270000, 128, 128  # 16 KiB a page
    k8, v8 = (torch.empty((pages, 1, page, dim), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((pages, 1), device="cuda") for _ in range(2))
    cache = avae.KvCacheQ8(k8, v8, ks, vs)
    table = np.array([[269999, 262200, 5]], np.int32)
    lens, cu = np.array([300], np.int32), np.array([0, 300], np.int32)
    rng = np.random.default_rng(11)
    k, v = (rng.normal(size=(300, 1, dim)).astype(np.float32) for _ in range(2))
    args = (_dev(table), _dev(cu), _dev(lens))
    avae.kv_write_q8(cache, _dev(k), _dev(v), *args)
    small = {p: i for i, p in enumerate(table[0])}
    t = np.array([[small[p] for p in table[0]]], np.int32)
    q = [np.zeros((3, 1, page, dim), np.int8) for _ in range(2)]
    s = [np.zeros((3, 1), np.float32) for _ in range(2)]
    for i, x in enumerate((k, v)):
        R.kv_write(q[i], s[i], x, t, cu, [300], 3, page)
    rk, rv = avae.kv_read_q8(cache, *args, total=300)
    assert np.array_equal(_np(rk), R.kv_read(q[0], s[0], t, cu, [300], page))
    assert np.array_equal(_np(rv), R.kv_read(q[1], s[1], t, cu, [300], page))
    for rows in (1, 300):
        one = np.array([0, rows], np.int32)
        x = rng.normal(size=(rows, 2, dim)).astype(np.float32)
        out = avae.attn_q8(_dev(x), cache, args[0], _dev(one), args[2])
        ref = R.attention(x, q[0], s[0], q[1], s[1], t, one, [300], page, dim ** -0.5)[0]
        assert np.abs(_np(out) - ref).max() <= 1e-4


def test_calls_in_a_captured_graph():
    """The calls allocate and synchronise nothing of their own: captured, and
    replayed with other work between the replays, they give the eager bits."""
    torch = _t()
    from bigvgan_waveform_decoder_amd import avae
    announce("8-bit operators in a graph")
    lens, new = [700, 90], [1, 33]
    c = Cache(34, lens, 2, 64, 16)
    dev = c.upload()
    cu = _cu(new)
    args = (_dev(c.table), _dev(cu), _dev(c.lens))
    rng = np.random.default_rng(5)
    x, w = _dev(rng.normal(size=(34, 256)).astype(np.float32)), _dev(np.ones(256, np.float32))
    pw, ps = avae.quant_q8(_dev(rng.normal(size=(8 * 64, 256)).astype(np.float32)))

    def run():
        q8, s, _ = avae.rms_norm_q8(x, w)
        y = avae.linear_q8(q8, s, pw, ps, act="silu", dtype=torch.bfloat16)
        q, k, v = y[:, :256], y[:, 256:384], y[:, 384:]
        avae.kv_write_q8(dev, k.unflatten(1, (2, 64)), v.unflatten(1, (2, 64)), *args, max_new=33)
        return avae.attn_q8(q.unflatten(1, (4, 64)), dev, *args, max_q=33, max_len=700)

    want = run().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for _ in range(3):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert torch.equal(run(), want)
