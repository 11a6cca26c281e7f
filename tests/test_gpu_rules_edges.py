"""Calls of the operators that turn heads and of the attention with rules as
programs make them: on other streams, captured, over caches past 32-bit
offsets, many sequences at once, offsets that do not lie in the rows."""
import ctypes

import numpy as np
import pytest

from tests import rules_reference as X
from tests.gpu_util import announce
from tests.test_gpu_attn_rules import _check, _parents, _slopes
from tests.test_gpu_q8 import U, Cache, _cu, _dev, _np, _t, _typed

pytestmark = pytest.mark.gpu


def _freq(half):
    return (10000.0 ** (-np.arange(half) / half)).astype(np.float32)


def _calls(avae, rng):
    """Each entry point once, by name: functions of a stream."""
    torch = _t()
    c = Cache(52, [9001, 300], 2, 64, 16)
    dev = c.upload()
    cu, cu1 = _dev(_cu([1, 40])), _dev(_cu([1, 1]))
    table, lens = _dev(c.table), _dev(c.lens)
    x = _dev(rng.normal(size=(41, 12, 64)).astype(np.float32))
    w, rope = _dev(np.ones(64, np.float32)), avae.Rope(_dev(_freq(32)))
    parents = _dev(_parents(rng, [1, 40]))
    mask, _ = avae.tree_mask(parents, cu, lens)
    # (inputs live as long as the calls: another stream still reads them)
    prefix, slopes = _dev(np.array([700, 100], np.int32)), _dev(_slopes(8))

    def write(s):
        avae.kv_write_rope_q8(dev, x[:, 8:10], x[:, 10:], table, cu, lens, rope, k_weight=w, stream=s)
        return avae.kv_read_q8(dev, table, cu, lens, 41, stream=s)

    return {
        "qk_norm_rope": lambda s: avae.qk_norm_rope(x[:, :8], x[:, 8:10], rope, w, w, cu=cu, lens=lens,
                                                    stream=s),
        "kv_write_rope_q8": write,
        "attn_rules_q8": lambda s: avae.attn_rules_q8(
            x[:, :8], dev, table, cu, lens, window=2000, cap=10.0, prefix=prefix, return_lse=True, stream=s),
        "attn_rules_q8, a row each": lambda s: avae.attn_rules_q8(
            x[:2, :8], dev, table, cu1, lens, max_q=1, slopes=slopes, stream=s),
        "attn_tree_q8": lambda s: avae.attn_tree_q8(x[:, :8], dev, table, cu, lens, mask, stream=s),
        "tree_mask": lambda s: avae.tree_mask(parents, cu, lens, stream=s)}


def test_stream_argument():
    """Calls on a stream other than the current one, which has work ahead of
    them: the same outputs, and what the current stream allocates right after
    is its own."""
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    side = torch.cuda.Stream()
    busy = torch.zeros(1 << 28, device="cuda")
    sizes = [41 * 8 * 64 * 4, 41 * 2 * 64 * 4, 41 * 8 * 4, 41 * 2 * 4, 41 * 4, 2 * 8 * 64 * 4]
    sizes += [41 * 8 * n * 68 * 4 for n in range(1, 40)] + [2 * 8 * n * 68 * 4 for n in range(60, 80)]
    for name, call in _calls(avae, np.random.default_rng(12)).items():
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


def test_calls_in_a_captured_graph():
    """Captured as a layer runs them, and replayed with eager calls of the same
    between the replays: the eager bits."""
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    announce("operators that turn heads, and the attention with rules, in a graph")
    calls = _calls(avae, np.random.default_rng(5))

    def run():
        out = []
        for call in calls.values():
            y = call(None)
            out += list(y) if isinstance(y, tuple) else [y]
        return out

    c = Cache(53, [700, 90], 2, 64, 16)
    dev = c.upload()
    cu, table, lens = _dev(_cu([1, 33])), _dev(c.table), _dev(c.lens)
    rng = np.random.default_rng(6)
    x = _dev(rng.normal(size=(34, 8, 64)).astype(np.float32))
    w, rope, bend = _dev(np.ones(64, np.float32)), avae.Rope(_dev(_freq(20)), True), _dev(_slopes(4))
    parents, prefix = _dev(_parents(rng, [1, 33])), _dev(np.array([50, 20], np.int32))

    def layer():
        mask, pos = avae.tree_mask(parents, cu, lens, max_rows=33)
        q, _ = avae.qk_norm_rope(x[:, :4], None, rope, w, positions=pos)
        avae.kv_write_rope_q8(dev, x[:, 4:6], x[:, 6:], table, cu, lens, rope, w, positions=pos, max_new=33)
        a = avae.attn_tree_q8(q, dev, table, cu, lens, mask, max_q=33, max_len=700)
        b = avae.attn_rules_q8(q, dev, table, cu, lens, max_q=33, max_len=700, cap=9.0, slopes=bend,
                               window=100, prefix=prefix, max_prefix=50)
        return mask, pos, q, a, b

    want = [t.clone() for t in layer()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = layer()
        graphs.append((g, got))
    first = [t.clone() for t in run()]
    for _ in range(3):
        for g, got in graphs:
            for t in got:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert all(torch.equal(a, b) for a, b in zip(layer(), want))
            assert all(torch.equal(a, b) for a, b in zip(run(), first))


def test_caches_past_32_bit_offsets():
    """Pages that start past 4 GiB: written with turned keys, and seen by rows
    of every kernel."""
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    announce("cache past 4 GiB with rules")
    heads, page, dim = 2, 64, 128
    n = (5 << 30) // (heads * page * dim)
    shape = (n, heads, page, dim)
    k8, v8 = (torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(shape[:2], device="cuda") for _ in range(2))
    cache = avae.KvCacheQ8(k8, v8, ks, vs)
    pages = np.array([[n - 1, 3, n - 7, n // 2 + 5, n - 300]], np.int32)
    rng = np.random.default_rng(8)
    k = rng.normal(size=(300, heads, dim)).astype(np.float32)
    v = rng.normal(size=(300, heads, dim)).astype(np.float32)
    table, lens = _dev(pages), _dev(np.array([300], np.int32))
    rope = avae.Rope(_dev(_freq(64)))
    avae.kv_write_rope_q8(cache, _dev(k), _dev(v), table, _dev(_cu([300])), lens, rope)
    want, size = X.turn(k, np.arange(300), _freq(64))
    got, _ = avae.kv_read_q8(cache, table, _dev(_cu([300])), lens, 300)
    top = np.abs(want).reshape(300, heads, dim).max((0, 2)).max() / 127
    assert np.abs(_np(got) - want).max() <= 0.51 * top
    at = pages[0]
    part = lambda t: _np(t[torch.from_numpy(at.astype(np.int64)).cuda()])
    p8, q8, ps, qs = part(k8), part(v8), part(ks), part(vs)
    mine = np.arange(5, dtype=np.int32)[None]
    for rows in (1, 20, 120):
        q, qf = _typed(rng.normal(size=(rows, 4, dim)), "f32")
        cu = _cu([rows])
        lines = X.lineage(_parents(rng, [rows]), cu)
        tree = _dev(X.tree_words(lines, -(-rows // 32)))
        pre = np.array([33], np.int32)
        a = avae.attn_tree_q8(q, cache, table, _dev(cu), lens, tree)
        b = avae.attn_rules_q8(q, cache, table, _dev(cu), lens, window=70, prefix=_dev(pre), cap=5.0)
        ra = X.attention(qf, p8, ps, q8, qs, mine, cu, [300], page, dim ** -0.5, lines=lines)[0]
        rb = X.attention(qf, p8, ps, q8, qs, mine, cu, [300], page, dim ** -0.5, window=70, prefix=pre,
                         cap=5.0)[0]
        assert np.abs(_np(a) - ra).max() <= 1e-4 and np.abs(_np(b) - rb).max() <= 1e-4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [0, 70])
def test_prompts_drafts_and_single_tokens_in_one_call(window, dtype):
    """The longest chooses the kernel for all."""
    new, lens = [200, 1, 33, 0, 7], [260, 900, 40, 10, 1000]
    announce(f"attn_rules_q8 {new} window {window} {dtype}")
    for heads, kv, dim in ((4, 2, 64), (2, 2, 128)):
        c = Cache(60, lens, kv, dim, 32)
        c.poison_unused()
        pre = np.array([70, 300, 50, 3, 0], np.int32)
        _check(c, new, heads, dtype, 1, window=window, prefix=pre, cap=8.0)
        _check(c, new, heads, dtype, 2, lines=X.lineage(_parents(np.random.default_rng(3), new), _cu(new)))


@pytest.mark.parametrize("rows", [1, 9, 20, 70])
def test_more_sequences_than_lanes(rows):
    """70 sequences: no chunk is chosen on the device for them."""
    announce(f"attn_tree_q8 70 sequences of {rows}")
    rng = np.random.default_rng(4)
    lens = [int(n) for n in rng.integers(rows, 400, size=70)]
    new = [int(rng.integers(0, rows + 1)) for _ in lens]
    c = Cache(61, lens, 2, 64, 16)
    c.poison_unused()
    _check(c, new, 4, "bf16", 1, lines=X.lineage(_parents(rng, new), _cu(new)), slack=rows)
    _check(c, new, 4, "bf16", 2, slopes=_slopes(4), slack=rows)


def test_the_same_bits_twice():
    announce("attn_rules_q8 twice")
    lens, new = [6000, 900, 3001], [30, 2, 70]
    c = Cache(62, lens, 2, 128, 64)
    q, _ = _typed(np.random.default_rng(3).normal(size=(102, 6, 128)), "bf16")
    tree = _dev(X.tree_words(X.lineage(_parents(np.random.default_rng(5), new), _cu(new)), 3))
    args = (q, c.upload(), _dev(c.table), _dev(_cu(new)), _dev(c.lens))
    first = c.avae.attn_tree_q8(*args, tree, max_q=70).clone()
    rules = c.avae.attn_rules_q8(*args, max_q=70, cap=5.0, slopes=_dev(_slopes(6))).clone()
    for _ in range(3):
        assert _t().equal(c.avae.attn_tree_q8(*args, tree, max_q=70), first)
        assert _t().equal(c.avae.attn_rules_q8(*args, max_q=70, cap=5.0, slopes=_dev(_slopes(6))), rules)


@pytest.mark.parametrize("rows", [4, 40, 100])
def test_offsets_that_do_not_lie_in_the_rows(rows):
    """cu that falls, or leaves the rows: those sequences have none; what lies
    behind the last one stays; lengths past the table add no key."""
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    announce(f"attn_rules_q8 bad offsets {rows}")
    L = avae.lib()
    c = Cache(63, [300, 300, 300], 2, 64, 16)
    cu = np.array([0, rows, 5000, rows], np.int32)
    lens = np.array([300, 300, 9999], np.int32)
    dev = c.upload()
    q, qf = _typed(np.random.default_rng(1).normal(size=(rows + 3, 4, 64)), "f32")
    tcu, tlens, table = _dev(cu), _dev(lens), _dev(c.table)
    tree = _dev(X.tree_words([[i] for i in range(rows + 3)], 4))
    for rules, kw in ((avae.avae_attn_rules(9.0, None, None, 0, None, 0, 0), dict(cap=9.0)),
                      (avae.avae_attn_rules(0.0, None, None, 0, tree.data_ptr(), 4, 4),
                       dict(lines=[[i] for i in range(rows)]))):
        out = torch.full((rows + 3, 4, 64), 7.0, device="cuda")
        ragged = avae.avae_ragged(tcu.data_ptr(), tlens.data_ptr(), table.data_ptr(), c.table.shape[1],
                                  c.table.shape[1], 3, rows + 3, rows)
        need = L.avae_attn_rules_q8_workspace_bytes(dev.ref, ctypes.addressof(ragged), 4, 0, 304, 0,
                                                    ctypes.addressof(rules))
        ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
        rc = L.avae_attn_rules_q8(q.data_ptr(), 256, 64, 4, 0, dev.ref, ctypes.addressof(ragged), None, 304,
                                  0.125, 1, 0, ctypes.addressof(rules), out.data_ptr(), None, ws.data_ptr(),
                                  need, None)
        assert rc == 0
        torch.cuda.synchronize()
        ref = X.attention(qf[:rows], c.k8, c.ks, c.v8, c.vs, c.table[:1], np.array([0, rows]), [300], 16,
                          0.125, **kw)[0]
        assert np.abs(_np(out)[:rows] - ref).max() <= 1e-4
        assert (_np(out)[rows:] == 7.0).all()


@pytest.mark.parametrize("rows", [1, 9, 40, 100, 300])
def test_bounds_on_lengths_far_past_them(rows):
    """max_len at the most that a table may cover, and short sequences: the
    chunks that it is cut into start past every key."""
    from bigvgan_waveform_decoder_amd import avae
    torch = _t()
    announce(f"attn_rules_q8 max_len 2^29, {rows} rows")
    lens = [700, 301]
    new = [rows, 1]
    c = Cache(64, lens, 2, 64, 256)
    c.poison_unused()
    wide = torch.full((2, 1 << 21), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = _dev(c.table)
    q, qf = _typed(np.random.default_rng(1).normal(size=(rows + 1, 4, 64)), "f32")
    dev, cu, n = c.upload(), _dev(_cu(new)), _dev(c.lens)
    tree = _dev(X.tree_words([[i] for i in range(rows)] + [[0]], 10))
    pre = np.array([100, 50], np.int32)
    for kw in (dict(cap=9.0), dict(window=70, prefix=pre), dict(window=1 << 28, prefix=pre), dict(lines=1)):
        if "lines" in kw:
            kw = dict(lines=[[i] for i in range(rows)] + [[0]])
            out = avae.attn_tree_q8(q, dev, wide, cu, n, tree, max_q=rows, max_len=1 << 29)
        else:
            on = {k: _dev(v) if isinstance(v, np.ndarray) else v for k, v in kw.items()}
            out = avae.attn_rules_q8(q, dev, wide, cu, n, max_q=rows, max_len=1 << 29, **on)
        ref = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, _cu(new), lens, 256, 0.125, **kw)[0]
        assert np.abs(_np(out) - ref).max() <= 1e-4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_rows_than_tokens_with_windows_and_prefixes(dtype):
    """Rows before their sequence's first token see nothing, not the prefix."""
    announce(f"attn_rules_q8 more rows than tokens {dtype}")
    for new, lens in (([5, 2], [3, 40]), ([40, 3], [30, 2]), ([150], [100]), ([3], [0])):
        c = Cache(65, lens, 2, 64, 16)
        c.poison_unused()
        for window in (0, 2, 64):
            _check(c, new, 4, dtype, 1, window=window, prefix=np.full(len(new), 7, np.int32), cap=5.0)
        _check(c, new, 4, dtype, 2, lines=X.lineage(_parents(np.random.default_rng(3), new), _cu(new)))


def test_factors_past_float32_under_a_cap():
    """Scales and caps whose quotient leaves float32: a key that the query has
    nothing in common with scores 0 all the same."""
    announce("attn_rules_q8 factors past float32")
    for new, lens in (([1], [200]), ([9], [200]), ([60], [200]), ([100], [300])):
        c = Cache(66, lens, 2, 64, 16)
        c.k8[:, :, ::3] = 0
        q = np.random.default_rng(1).normal(size=(sum(new), 4, 64))
        for scale, cap, gain in ((1e30, 1e-30, 1.0), (1.0, 1e-30, 2.0 ** 120), (-1e30, 1e-30, 1e10)):
            qf = (q * gain).astype(np.float32)
            out = c.avae.attn_rules_q8(_dev(qf), c.upload(), _dev(c.table), _dev(_cu(new)), _dev(c.lens),
                                       scale=scale, cap=cap)
            # (scores within 1e-30 of each other: the mean of the values)
            ref = X.attention(qf, c.k8, c.ks, c.v8, c.vs, c.table, _cu(new), lens, 16, scale, cap=cap)[0]
            assert np.abs(_np(out) - ref).max() <= 1e-4


@pytest.mark.parametrize("rows", [1, 40])
def test_windows_and_prefixes_past_32_bits(rows):
    """Bounds that no 32-bit number holds: as the largest that one does, not as
    their low bits."""
    rng = np.random.default_rng(21)
    c = Cache(53, [900, 300], 2, 64, 16)
    c.upload()
    q = _typed(rng.normal(size=(2 * rows, 8, 64)), "f32")[0]
    args = (q, c.dev, _dev(c.table), _dev(_cu([rows, rows])), _dev(c.lens))
    announce(f"attn_rules_q8 window, max_prefix past 32 bits, {rows} rows")
    avae = c.avae
    prefix = _dev(np.array([700, 200], np.int32))
    whole = avae.attn_rules_q8(*args, max_q=rows, cap=10.0)
    assert _t().equal(whole, avae.attn_rules_q8(*args, max_q=rows, cap=10.0, window=2 ** 32 + 3))
    near = avae.attn_rules_q8(*args, max_q=rows, window=50, prefix=prefix, max_prefix=2 ** 31 - 1)
    far = avae.attn_rules_q8(*args, max_q=rows, window=50, prefix=prefix, max_prefix=2 ** 32 + 3)
    assert _t().equal(near, far)
    with pytest.raises(avae.AvaeError):
        avae.attn_rules_q8(*args, max_q=rows, max_len=2 ** 32 + 3)
