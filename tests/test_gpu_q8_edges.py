"""The 8-bit serving operators where keys are split, ranges are wide, calls are
padded and streams are mixed, against the plain numpy forms."""
import numpy as np
import pytest

from tests import q8_reference as R
from tests.gpu_util import announce
from tests.test_gpu_q8 import ROUND, U, Cache, _cu, _dev, _dtype, _np, _t, _typed

pytestmark = pytest.mark.gpu


def _attend(c, new, qf, dtype, causal=True, window=0, first=None, **kw):
    """(out, lse, reference out, reference lse, tolerance) of float64 queries."""
    cu = _cu(new)
    dq, qf = _typed(qf, dtype)
    out, lse = c.avae.attn_q8(dq, c.upload(), _dev(c.table), _dev(cu), _dev(c.lens), causal=causal,
                              window=window, first=None if first is None else _dev(first),
                              return_lse=True, **kw)
    with np.errstate(invalid="ignore"):
        ref, rlse, weight, size = R.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, cu, list(c.lens),
                                              c.page, c.dim ** -0.5, causal, window, first)
    # Score: dim float32 additions and a few roundings, 22 bits of a float32
    # query; probabilities: the score's error, their own rounding (11 or 22
    # bits), the sums over the keys; float16's smallest step is 2^-40 of the
    # row's largest value scale, which is at most the largest of the call.
    length = max(c.lens)
    ds = (c.dim + 16) * U * size + (2.0 ** -21 * size if dtype == "f32" else 0)
    dp = 2 * np.expm1(ds) + (length / 8 + 64) * U + (2.0 ** -21 if dtype == "f32" else 2.0 ** -11)
    rel, step = ROUND[dtype]
    tol = dp[:, :, None] * weight + rel * np.abs(ref) + step
    return _np(out), _np(lse), ref, rlse, tol


# new, lengths, heads, cache heads, dim: few and many rows, each with either join
SPLIT = [([1], [2400], 4, 2, 64), ([1], [2400], 4, 2, 128), ([2], [1300], 2, 1, 256),
         ([1] * 32, [600] * 31 + [410], 64, 2, 64), ([1] * 32, [500] * 32, 64, 2, 128),
         ([100], [1500], 8, 2, 64), ([70], [1100], 4, 2, 128), ([260], [1300], 8, 1, 64),
         ([260], [1400], 8, 1, 128)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens,heads,kv_heads,dim", SPLIT)
@pytest.mark.parametrize("what", ["query", "k page", "v page", "k pages", "v pages"])
def test_nan_stays_where_keys_are_split(what, new, lens, heads, kv_heads, dim, dtype):
    """A NaN query row, a NaN page as long as a chunk and caches of nothing
    else: exactly the rows that see one are NaN, however the keys are cut."""
    announce(f"attn_q8 NaN {what}, split keys {new[:3]} {lens[:3]} {heads}/{kv_heads} dim {dim} {dtype}")
    c = Cache(50, lens, kv_heads, dim, 128)
    c.poison_unused()
    rng = np.random.default_rng(3)
    q = rng.normal(size=(sum(new), heads, dim)) * 2
    if what == "query":
        q[0, heads - 1, 5] = np.nan
    scales = c.vs if what[0] == "v" else c.ks
    if "page" in what:
        scales[c.table[0, 2 if what.endswith("page") else slice(0, -(-lens[0] // 128))],
               kv_heads - 1] = np.nan
    out, lse, ref, rlse, tol = _attend(c, new, q, dtype)
    bad = np.isnan(ref).any(2)
    assert bad.any() and np.array_equal(np.isnan(ref).all(2), bad)
    assert np.array_equal(np.isnan(out), np.isnan(ref)) and np.array_equal(np.isnan(lse), bad)
    assert np.all(np.abs(out - ref)[~bad] <= tol[~bad])
    assert np.all(np.abs(lse - rlse)[~bad] <= 1e-3)


# heads of 64, 128 and 256 dims: 4, 2 and 1 chunks a wave and step
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,total", [(4, 4, 64, 512), (4, 2, 128, 600),
                                                      (2, 1, 256, 1100)])
@pytest.mark.parametrize("length", [300, 2050, 2600, 4170, 5249, 8190])
def test_packed_rows_longer_than_the_sequences(length, heads, kv_heads, dim, total, dtype):
    """Packed tensors with rows that belong to no sequence, which choose the
    join for many rows: any number of chunks, odd ones among them."""
    announce(f"attn_q8 padded total {total}, {length} keys {heads}/{kv_heads} dim {dim} {dtype}")
    c = Cache(51, [length], kv_heads, dim, 64)
    c.poison_unused()
    rng = np.random.default_rng(5)
    q = rng.normal(size=(total, heads, dim)) * 2
    dq, _ = _typed(q, dtype)
    got, glse = c.avae.attn_q8(dq, c.upload(), _dev(c.table), _dev(_cu([1])), _dev(c.lens), max_q=1,
                               return_lse=True)
    out, lse, ref, rlse, tol = _attend(c, [1], q[:1], dtype)  # the row alone: joined otherwise
    for o, l in ((out, lse), (_np(got)[:1], _np(glse)[:1])):
        assert np.all(np.abs(o - ref) <= tol)
        assert np.all(np.abs(l - rlse) <= 1e-3)


def test_stream_argument():
    """Calls on a stream other than the current one, which has work ahead of
    them: what the current stream allocates right after the call returns is
    its own, whether the outputs are kept or dropped."""
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    rng = np.random.default_rng(12)
    c = Cache(52, [9001], 2, 64, 16)
    dev = c.upload()
    one, back = _dev(_cu([1])), _dev(_cu([800]))
    table, lens = _dev(c.table), _dev(c.lens)
    x, w = _dev(rng.normal(size=(1000, 500)).astype(np.float32)), _dev(np.ones(500, np.float32))
    a, sa = avae.quant_q8(_dev(rng.normal(size=(1000, 77)).astype(np.float32)))
    b, sb = avae.quant_q8(_dev(rng.normal(size=(900, 77)).astype(np.float32)))
    q = _dev(rng.normal(size=(1, 8, 64)).astype(np.float32))
    kv = _dev(rng.normal(size=(1, 2, 64)).astype(np.float32))
    assert avae.lib().avae_linear_q8_workspace_bytes(1000, 900, 77) > 0

    def write(s):
        avae.kv_write_q8(dev, kv, kv, table, one, lens, stream=s)
        return avae.kv_read_q8(dev, table, one, lens, 1, stream=s)

    calls = {
        "rms_norm_q8": lambda s: avae.rms_norm_q8(x, w, residual=x, stream=s),
        "quant_q8": lambda s: avae.quant_q8(x, stream=s),
        "dequant_q8": lambda s: avae.dequant_q8(a, sa, stream=s),
        "linear_q8": lambda s: avae.linear_q8(a, sa, b, sb, stream=s),
        "kv_write_q8": write,
        "kv_read_q8": lambda s: avae.kv_read_q8(dev, table, back, lens, 800, stream=s),
        "attn_q8": lambda s: avae.attn_q8(q, dev, table, one, lens, return_lse=True, stream=s)}
    side = torch.cuda.Stream()
    busy = torch.zeros(1 << 28, device="cuda")
    # workspaces and outputs of these calls, in bytes
    sizes = [avae.lib().avae_linear_q8_workspace_bytes(1000, 900, 77), 1000 * 900 * 4, 1000 * 500 * 4,
             1000 * 500, 1000 * 77 * 4, 4000, 800 * 128 * 4, 512, 2048]
    sizes += [8 * n * 68 * 4 for n in range(60, 80)]  # parts of the attention, whatever their number

    for name, call in calls.items():
        announce(f"{name} on a stream of its own")
        as_list = lambda y: list(y) if isinstance(y, tuple) else [y]
        want = [t.clone() for t in as_list(call(None))]
        torch.cuda.synchronize()
        for keep in (True, False):
            with torch.cuda.stream(side):
                for _ in range(10):
                    busy.add_(1)
            out = as_list(call(side))
            if not keep:
                del out
            marks = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in 2 * sizes]
            torch.cuda.synchronize()
            assert all(bool((m == 0x55).all()) for m in marks)
            if keep:
                assert all(torch.equal(g, t) for g, t in zip(out, want))


@pytest.mark.parametrize("eps", [0.0, 1e-35, 1e-6])
@pytest.mark.parametrize("C", [1, 5, 500, 1536, 9000, 33001])
def test_norm_rows_scales_over_the_whole_range(C, eps):
    """Rows of zeros, rows whose squares pass float32's largest number or fall
    below its smallest, and ordinary ones beside them."""
    from bigvgan_waveform_decoder_amd import avae
    announce(f"rms_norm_q8 range C={C} eps={eps}")
    rng = np.random.default_rng(C)
    tops = [0, 1e-44, 3e-39, 1e-30, 1e-22, 1e-12, 1.0, 1e15, 1e19, 1e20, 1e30, 1e37]
    x = rng.normal(size=(len(tops), C))
    x = (x / np.abs(x).max(1, keepdims=True) * np.array(tops)[:, None]).astype(np.float32)
    r = (x * rng.normal(size=x.shape) * 0.1).astype(np.float32)
    w = (1 + 0.2 * rng.normal(size=C)).astype(np.float32)
    for res in (None, r):
        q, s, _ = avae.rms_norm_q8(_dev(x), _dev(w), eps=eps, residual=None if res is None else _dev(res))
        with np.errstate(invalid="ignore"):
            rq, rs, _ = R.rows_q8(x, w, res, float(np.float32(eps)))
        rs[np.abs(rq).max(1) == 0] = 0
        assert rs[0] == 0 and np.isfinite(rs).all()
        got = _np(s).astype(np.float64)
        assert np.array_equal(_np(q), rq)
        # C/256 terms a lane and a few roundings; float32's smallest step
        assert np.all(np.abs(got - rs) <= (C / 256 + 24) * U * rs + 2.0 ** -149), (got, rs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cache_read_of_sequences_without_tokens(dtype):
    """Rows of a sequence of length 0 (or below) are zeros, rows of none stay."""
    import ctypes
    from bigvgan_waveform_decoder_amd import avae
    announce(f"kv_read_q8 lengths of 0 {dtype}")
    torch = _t()
    c = Cache(53, [20, 0, 40, 0], 2, 64, 16)
    dev = c.upload()
    c.lens[3] = -5
    new = [20, 3, 2, 4]
    table, cu, lens = _dev(c.table), _dev(_cu(new)), _dev(c.lens)
    k, v = (torch.full((31, 2, 64), 7.0, dtype=_dtype(dtype), device="cuda") for _ in range(2))
    rows = avae.avae_ragged(cu.data_ptr(), lens.data_ptr(), table.data_ptr(), c.table.shape[1],
                            c.table.shape[1], 4, 31, 20)
    assert avae.lib().avae_kv_read_q8(dev.ref, ctypes.byref(rows), {"f32": 0, "bf16": 1}[dtype],
                                      k.data_ptr(), v.data_ptr(),
                                      torch.cuda.current_stream().cuda_stream) == 0
    before = _np(dev.k).copy(), _np(dev.k_scale).copy()
    for got, q8, s in ((k, c.k8, c.ks), (v, c.v8, c.vs)):
        want = R.kv_read(q8, s, c.table, _cu(new), [20, 0, 40, 0], 16)
        want = torch.from_numpy(want).to(_dtype(dtype)).float().numpy()
        assert (want[20:23] == 0).all() and (want[25:29] == 0).all() and (want[23:25] != 0).any()
        assert np.array_equal(_np(got)[:29], want) and (_np(got)[29:] == 7).all()
    # and a write of such rows changes nothing
    x = torch.ones((29, 2, 64), device="cuda")
    only = _dev(np.array([0, 0, 3, 3, 7], np.int32))
    avae.kv_write_q8(dev, x, x, table, only, lens)
    assert np.array_equal(_np(dev.k), before[0]) and np.array_equal(_np(dev.k_scale), before[1])


def _scaled_cache(seed, lens, heads, dim, page, low, high, zeros):
    """Value scales 2^low .. 2^high, a page each; every fifth page of zeros if asked for."""
    c = Cache(seed, lens, heads, dim, page)
    c.poison_unused()
    rng = np.random.default_rng(seed)
    for b, t in enumerate(lens):
        for col in range(-(-t // page)):
            p = c.table[b, col]
            c.vs[p] = np.exp2(rng.integers(low, high + 1)).astype(np.float32)
            if zeros and col % 5 == 3:
                c.vs[p], c.v8[p] = 0, 0
    return c


def _check_scaled(c, new, heads, dtype, q):
    out, lse, ref, rlse, tol = _attend(c, new, q, dtype)
    # float16's smallest step: 2^-40 of the largest value scale for each key;
    # the smallest bfloat16 step of outputs near float32's own end
    top = c.vs[c.table[c.table >= 0]].max()
    tol = tol + 2.0 ** -40 * 127 * max(c.lens) * top + 2.0 ** -133
    assert np.all(np.abs(out - ref) <= tol), (np.abs(out - ref) / tol).max()
    assert np.all(np.abs(lse - rlse) <= 1e-3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,dim", [(2, 64), (4, 128), (2, 256)])
@pytest.mark.parametrize("new,lens", [([100, 70, 64, 40], [200, 200, 64, 130]), ([90], [1300])])
def test_many_rows_over_small_and_distant_value_scales(new, lens, heads, dim, dtype):
    """Value scales down to float32's smallest normal number, scales far apart,
    pages of zeros: many rows, whole and split."""
    rng = np.random.default_rng(9)
    q = rng.normal(size=(sum(new), heads, dim))
    q[0] *= 1e-30
    q[1] *= 30
    q[2] = 0
    for low, high, zeros in ((-126, -126, False), (-125, -112, True), (-112, -90, False),
                             (-20, 10, True), (60, 90, False)):
        announce(f"attn_q8 many rows, value scales 2^{low}..2^{high} {new} {lens} dim {dim} {dtype}")
        _check_scaled(_scaled_cache(61, lens, 2, dim, 16, low, high, zeros), new, heads, dtype, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,dim", [(2, 64), (4, 128), (2, 256)])
@pytest.mark.parametrize("new,lens", [([1, 2, 8], [200, 64, 130]), ([3], [1300])])
def test_few_rows_over_small_and_distant_value_scales(new, lens, heads, dim, dtype):
    """The same with few rows, below float32's smallest normal number as well."""
    rng = np.random.default_rng(9)
    q = rng.normal(size=(sum(new), heads, dim))
    q[0] *= 1e-30
    q[1] *= 30
    q[2] = 0
    for low, high, zeros in ((-140, -132, False), (-126, -126, False), (-125, -112, True),
                             (-112, -90, False), (-20, 10, True), (60, 90, False)):
        announce(f"attn_q8 few rows, value scales 2^{low}..2^{high} {new} {lens} dim {dim} {dtype}")
        _check_scaled(_scaled_cache(62, lens, 2, dim, 16, low, high, zeros), new, heads, dtype, q)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens,window,growth", [
    ([2], [17], 0, 50), ([4], [28], 10, -50), ([3, 1, 2], [34, 20, 16], 0, 40),  # few rows
    ([70], [70], 0, 25), ([70], [70], 20, -25), ([100], [700], 30, 3), ([100], [700], 30, -3),
    ([260], [700], 40, -4)])
@pytest.mark.parametrize("dim", [64, 128])
def test_scales_of_pages_that_only_other_rows_see(new, lens, window, growth, dim, dtype):
    """Value scales that grow or fall from page to page by a power of two:
    every row keeps its bits relative to the pages that it sees itself."""
    announce(f"attn_q8 others' pages {new} {lens} window {window} 2^{growth} a page dim {dim} {dtype}")
    c = Cache(63, lens, 1, dim, 16)
    c.poison_unused()
    for b, t in enumerate(lens):
        cols = np.arange(-(-t // 16))
        steps = cols if growth > 0 else cols[-1] - cols
        c.vs[c.table[b, cols], 0] = np.exp2(abs(growth) * steps - 60.0).astype(np.float32)
    rng = np.random.default_rng(4)
    q = rng.normal(size=(sum(new), 2, dim))
    out, lse, ref, rlse, tol = _attend(c, new, q, dtype, window=window)
    # float16's smallest step: 2^-40 of the largest value scale that the row sees
    cu = _cu(new)
    for b, t in enumerate(lens):
        for i in range(new[b]):
            pos = t - new[b] + i
            seen = np.arange((max(0, pos - window + 1) if window else 0) // 16, pos // 16 + 1)
            tol[cu[b] + i] += 2.0 ** -40 * 127 * t * c.vs[c.table[b, seen], 0].max()
    assert np.all(np.abs(out - ref) <= tol), (np.abs(out - ref) / tol).max()
    assert np.all(np.abs(lse - rlse) <= 1e-3)


def test_rows_past_one_launch():
    """2^26 rows and a few: more than one launch has threads for."""
    from bigvgan_waveform_decoder_amd import avae
    announce("quant_q8, rms_norm_q8, dequant_q8 of 2^26 + 9 rows")
    torch = _t()
    M, C = (1 << 26) + 9, 16
    x = torch.zeros((M, C), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, (1 << 21) - 1, 1 << 21, (1 << 24) + 3, 1 << 26, M - 2, M - 1], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    x[at] = torch.randn((len(at), C), device="cuda", generator=g).bfloat16()
    w = torch.rand(C, device="cuda", generator=g)
    for call in (avae.quant_q8, lambda t: avae.rms_norm_q8(t, w, residual=t)):
        got, want = call(x), call(x[at])
        for a, b in zip(got, want):
            if b is not None:
                assert torch.equal(a[at], b)
        q, s = got[:2]
        assert int((s != 0).sum()) == len(at) and int((q != 0).sum()) == int((q[at] != 0).sum())
        y = avae.dequant_q8(q, s, dtype=torch.bfloat16)
        assert torch.equal(y[at], avae.dequant_q8(q[at], s[at], dtype=torch.bfloat16))
        assert int((y != 0).sum()) == int((y[at] != 0).sum())
        del got, q, s, y


def test_linear_of_more_columns_than_a_launch_packs():
    """2^26 weight rows of odd length, laid out anew in one call."""
    from bigvgan_waveform_decoder_amd import avae
    announce("linear_q8 17 x 2^26 x 17")
    torch = _t()
    M, N, K = 17, (1 << 26) + 5, 17
    assert avae.lib().avae_linear_q8_workspace_bytes(M, N, K) > 0
    g = torch.Generator(device="cuda").manual_seed(5)
    a = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    one = torch.ones(M, device="cuda")
    y = avae.linear_q8(a, one, w, torch.ones(N, device="cuda"), dtype=torch.bfloat16)
    at = torch.cat([torch.arange(64), torch.arange(N - 200, N), torch.randint(0, N, (2000,))]).cuda()
    want = (a.cpu().double() @ w[at].cpu().double().t()).bfloat16()
    assert torch.equal(y[:, at].cpu(), want)


def test_bounds_on_rows_far_past_them():
    """max_rows and total of 2^28 where a sequence has a few rows: the write and
    the read of the cache go by what there is."""
    import ctypes
    from bigvgan_waveform_decoder_amd import avae
    announce("kv_write_q8, kv_read_q8 with bounds of 2^28 rows")
    torch = _t()
    new, lens = [20, 3], [50, 3]
    c = Cache(54, lens, 2, 64, 16)
    dev, cu = c.upload(), _cu([20, 3])
    table, dcu, dlens = _dev(c.table), _dev(cu), _dev(c.lens)
    rng = np.random.default_rng(1)
    x = rng.normal(size=(23, 2, 64)).astype(np.float32)
    dx = _dev(x)
    rows = avae.avae_ragged(dcu.data_ptr(), dlens.data_ptr(), table.data_ptr(), c.table.shape[1],
                            c.table.shape[1], 2, 1 << 28, 1 << 28)
    stream = torch.cuda.current_stream().cuda_stream
    L = avae.lib()
    assert L.avae_kv_write_q8(dx.data_ptr(), 128, 64, dx.data_ptr(), 128, 64, 0, dev.ref,
                              ctypes.byref(rows), stream) == 0
    for q8, s in ((c.k8, c.ks), (c.v8, c.vs)):
        R.kv_write(q8, s, x, c.table, cu, lens, c.n, 16)
    assert c.same()
    k, v = (torch.full((23, 2, 64), 7.0, device="cuda") for _ in range(2))
    assert L.avae_kv_read_q8(dev.ref, ctypes.byref(rows), 0, k.data_ptr(), v.data_ptr(), stream) == 0
    assert np.array_equal(_np(k), R.kv_read(c.k8, c.ks, c.table, cu, lens, 16))
    assert np.array_equal(_np(v), R.kv_read(c.v8, c.vs, c.table, cu, lens, 16))


@pytest.mark.parametrize("M,N", [(3, 512), (600, 640), (1500, 2048)])
def test_silu_in_float32_to_its_last_bits(M, N):
    """Exact sums with power-of-two scales: what is left is SiLU's own error, an
    exponential within one last place, an addition and a division.  Below -88 the
    exponential is past float32 and the value, under 3e-37, is 0."""
    from bigvgan_waveform_decoder_amd import avae
    announce(f"linear_q8 SiLU float32 {M}x{N}")
    torch = _t()
    rng = np.random.default_rng(N)
    a = rng.integers(-127, 128, size=(M, 64)).astype(np.int8)
    w = rng.integers(-127, 128, size=(N, 64)).astype(np.int8)
    a[0] = w[0]
    sw = np.exp2(rng.integers(-14, -9, size=N)).astype(np.float32)
    y = avae.linear_q8(_dev(a), torch.ones(M, device="cuda"), _dev(w), _dev(sw), act="silu")
    raw = R.linear_q8(a, np.ones(M, np.float32), w, sw)
    assert raw.min() < -80 and raw.max() > 80 and np.array_equal(raw, raw.astype(np.float32))
    ref = R.linear_q8(a, np.ones(M, np.float32), w, sw, act="silu")
    assert np.all(np.abs(_np(y) - ref) <= 6 * U * np.abs(ref) + 3e-37)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_silu_to_where_its_exponential_ends(dtype):
    """From -89 to -80: bfloat16 outputs end where float32's do."""
    from bigvgan_waveform_decoder_amd import avae
    announce(f"linear_q8 SiLU around -88 {dtype}")
    torch = _t()
    a = torch.ones((1, 64), dtype=torch.int8, device="cuda")
    w = torch.zeros((577, 64), dtype=torch.int8, device="cuda")
    v = torch.arange(577, device="cuda") / 64 - 89.0  # exact: -80 and a bias
    w[:, 0] = -80
    y = avae.linear_q8(a, torch.ones(1, device="cuda"), w, torch.ones(577, device="cuda"), bias=v + 80,
                       act="silu", dtype=_dtype(dtype))[0].double()
    v = v.double()
    ref = v / (1 + torch.exp(-v))
    rel, _ = ROUND[dtype]
    assert bool(((y - ref).abs() <= (rel + (6 * U if dtype == "f32" else 2.0 ** -16)) * ref.abs() + 3e-37).all())


# M, N, K, first column and columns left over of wider tensors: a tile kernel each
TILES = [(512, 1541, 400, 0, 0), (512, 1536, 256, 0, 0), (700, 1100, 112, 16, 32),  # 64 x 64
         (2000, 2500, 1552, 0, 0), (1500, 4100, 64, 0, 16),                         # 64 x 128
         (6000, 6144, 1536, 0, 0), (5900, 6200, 688, 0, 0),                         # 192 x 256, in rounds
         (4096, 4096, 320, 0, 0), (8000, 8100, 272, 0, 0),                          # 256 x 256, in rounds
         (600, 1541, 416, 3, 2), (2000, 2500, 208, 0, 1), (520, 1600, 48, 1, 0),    # through registers
         (1000, 1000, 77, 0, 0), (2100, 2300, 1001, 5, 2), (4096, 4096, 300, 0, 0)]  # laid out anew


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K,at,pad", TILES)
def test_linear_tiles(M, N, K, at, pad, dtype):
    """Sums that float32 holds: plain outputs have to be equal, SiLU's within
    its own error (an exponential, an addition and a division; 2^-16 quick)."""
    from bigvgan_waveform_decoder_amd import avae
    announce(f"linear_q8 tiles {M}x{N}x{K} at {at} pad {pad} {dtype}")
    torch = _t()
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, w = (torch.randint(-127, 128, (r, at + K + pad), dtype=torch.int8, device="cuda", generator=g)
            for r in (M, N))
    sa = torch.exp2(torch.randint(-4, 1, (M,), device="cuda", generator=g).float())
    sw = torch.exp2(torch.randint(-11, -8, (N,), device="cuda", generator=g).float())
    bias = torch.randint(-64, 65, (N,), device="cuda", generator=g) / 64.0
    a, w = a[:, at:at + K], w[:, at:at + K]
    raw = torch.mm(a.double(), w.t().double().contiguous()) * sa.double()[:, None] * sw.double()
    y = avae.linear_q8(a, sa, w, sw, dtype=_dtype(dtype))
    assert torch.equal(y, raw.to(_dtype(dtype)))
    del y
    y = avae.linear_q8(a, sa, w, sw, bias=bias, act="silu", dtype=_dtype(dtype)).double()
    raw += bias.double()
    assert torch.equal(raw, raw.float().double())
    raw /= 1 + torch.exp(-raw)
    rel, step = ROUND[dtype]
    rel += 6 * U if dtype == "f32" else 2.0 ** -16
    assert bool(((y - raw).abs() <= rel * raw.abs() + step + 3e-37).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("new,lens", [([2], [300]), ([90], [200])])
@pytest.mark.parametrize("power", [-110, -60, 60, 119, 121, 124, 125])
def test_queries_over_the_whole_range(power, new, lens, dtype):
    """Queries times a power of two, the softmax's scale over it: the same
    attention, up to float32's largest numbers."""
    announce(f"attn_q8 queries times 2^{power} {new} {lens} {dtype}")
    c = Cache(55, lens, 2, 64, 32)
    c.poison_unused()
    rng = np.random.default_rng(6)
    q = np.clip(rng.normal(size=(sum(new), 4, 64)), -3.9, 3.9)
    cu = _cu(new)
    dq, qf = _typed(q * 2.0 ** power, dtype)
    assert np.isfinite(qf).all()
    out = _np(c.avae.attn_q8(dq, c.upload(), _dev(c.table), _dev(cu), _dev(c.lens),
                             scale=0.125 * 2.0 ** -power))
    want, _, _, _, tol = _attend(c, new, q, dtype)  # dim 64: its own scale is 0.125
    assert np.all(np.abs(out - want) <= tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (6, 2, 128), (2, 2, 256)])
@pytest.mark.parametrize("window", [0, 700])
def test_prompt_and_single_tokens_in_one_call(window, heads, kv_heads, dim, dtype):
    """A prompt, drafts and single tokens over long keys, packed together; the
    same call again gives the same bits."""
    announce(f"attn_q8 mixed {heads}/{kv_heads} dim {dim} window {window} {dtype}")
    new, lens = [1, 300, 1, 0, 1, 7], [3000, 340, 2500, 90, 1, 1900]
    c = Cache(56, lens, kv_heads, dim, 64)
    c.poison_unused()
    rng = np.random.default_rng(7)
    q = rng.normal(size=(sum(new), heads, dim)) * 2
    first = np.array([5, 0, 2400, 0, 0, 100], np.int32)
    for f in (None, first):
        out, lse, ref, rlse, tol = _attend(c, new, q, dtype, window=window, first=f)
        assert np.all(np.abs(out - ref) <= tol)
        assert np.all(np.abs(lse - rlse) <= 1e-3)
        again, lse2 = _attend(c, new, q, dtype, window=window, first=f)[:2]
        assert np.array_equal(out, again) and np.array_equal(lse, lse2)
    # the single tokens alone
    for b, row in ((0, 0), (2, 301), (4, 302)):
        one = [int(i == b) for i in range(len(new))]
        out = _attend(c, one, q[row:row + 1], dtype, window=window, first=first)[0]
        assert np.all(np.abs(out - ref[row:row + 1]) <= tol[row:row + 1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new,lens", [([1, 2], [700, 350]), ([1], [4000]), ([90], [600]), ([40], [1300])])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_error_is_its_outputs_rounding(dim, new, lens, dtype):
    """Root mean square over an output: a correctly rounded result's error, and a
    tenth more for all that comes before the rounding."""
    announce(f"attn_q8 error {new} {lens} dim {dim} {dtype}")
    c = Cache(57, lens, 2, dim, 64)
    c.poison_unused()
    rng = np.random.default_rng(8)
    q = rng.normal(size=(sum(new), 8, dim))
    out, _, ref, _, _ = _attend(c, new, q, dtype)
    best = _t().from_numpy(ref).to(_dtype(dtype)).double().numpy()
    assert np.sqrt(np.mean((out - ref) ** 2)) <= 1.1 * np.sqrt(np.mean((best - ref) ** 2))
