"""Refusals of the operators that turn heads and of the attention with rules
(a code and a message before anything touches a device), and the frequencies,
which are made on the host."""
import ctypes

import numpy as np
import pytest

from bigvgan_waveform_decoder_amd import avae
from tests import rules_reference as X

EINVAL, ESHAPE, EWORKSPACE = -1, -2, -3
A, B, C, D = (ctypes.c_void_p(v) for v in (0x10000, 0x20000, 0x30000, 0x40000))
ODD = ctypes.c_void_p(0x10001)


def _p(struct):
    return None if struct is None else ctypes.addressof(struct)


def _message(who):
    assert avae.lib().avae_last_error().startswith(who.encode() + b": ")


# ------------------------------------------------------------------ frequencies

@pytest.mark.parametrize("scaling,kw", [
    ("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
    ("bands", dict(factor=8.0, context=8192.0, low=1.0, high=4.0)),
    ("ramp", dict(factor=16.0, context=4096.0, low=1.0, high=32.0)),
    ("ramp", dict(factor=2.0, context=100.0, low=20.0, high=21.0)), ("bands", dict(factor=1.0))])
@pytest.mark.parametrize("rot,theta", [(4, 10000.0), (64, 500000.0), (128, 10000.0), (50, 1.5)])
def test_frequencies(rot, theta, scaling, kw):
    """Both in 64 bits, rounded to float32 once: half a step, and 2^-24 more
    where the two powers differ in their last bits."""
    got, amp = avae.rope_freq(rot, theta, scaling, **kw)
    want, wamp = X.rope_freq(rot, theta, scaling, **kw)
    assert got.dtype == np.float32 and got.shape == (rot // 2,)
    assert np.all(np.abs(got - want) <= 2.0 ** -23 * want)
    assert abs(amp - wamp) <= 2.0 ** -24 * wamp
    assert got[0] <= 1.0 and np.all(np.diff(got) < 0)


@pytest.mark.parametrize("kw,code", [
    (dict(rot=0), ESHAPE), (dict(rot=7), ESHAPE), (dict(rot=1 << 17), ESHAPE), (dict(theta=1.0), EINVAL),
    (dict(theta=float("inf")), EINVAL), (dict(theta=float("nan")), EINVAL),
    (dict(scaling="linear", factor=0.5), EINVAL), (dict(scaling="linear", factor=float("nan")), EINVAL),
    (dict(scaling="base", rot=2, factor=2.0), ESHAPE), (dict(scaling="bands", context=0.0), EINVAL),
    (dict(scaling="bands", low=4.0, high=4.0), EINVAL), (dict(scaling="ramp", low=0.0), EINVAL),
    (dict(scaling="ramp", high=float("inf")), EINVAL)])
def test_frequency_refusals(kw, code):
    with pytest.raises(avae.AvaeError) as e:
        avae.rope_freq(**{**dict(rot=64, factor=2.0), **kw})
    assert e.value.code == code
    _message("avae_rope_freq")


def test_unknown_scaling():
    with pytest.raises(ValueError):
        avae.rope_freq(64, scaling="other")
    assert avae.lib().avae_rope_freq(64, 1e4, 5, 1.0, 1.0, 1.0, 2.0, A, B) == EINVAL
    assert avae.lib().avae_rope_freq(64, 1e4, 0, 1.0, 1.0, 1.0, 2.0, None, B) == EINVAL


# ------------------------------------------------------------------ heads

def _rope(freq=A, rot=64, interleaved=0, amp=1.0):
    return avae.avae_rope(freq, rot, interleaved, amp)


def _rows(cu=A, lens=B, table=C, ld=4, cols=4, seqs=2, total=10, max_rows=5):
    return avae.avae_ragged(cu, lens, table, ld, cols, seqs, total, max_rows)


DEFAULT = object()


def _qk(q=A, q_tok=256, q_head=64, heads=4, qw=B, k=C, k_tok=128, k_head=64, k_heads=2, kw=D, dim=64,
        dtype=1, eps=1e-6, rope=DEFAULT, pos=None, rows=DEFAULT, total=10, qo=B, qo_tok=256, qo_head=64,
        ko=D, ko_tok=128, ko_head=64):
    rope = _rope() if rope is DEFAULT else rope
    rows = _rows(table=None, ld=0, cols=0) if rows is DEFAULT else rows
    return avae.lib().avae_qk_norm_rope(q, q_tok, q_head, heads, qw, k, k_tok, k_head, k_heads, kw,
                                        dim, dtype, eps, _p(rope), pos, _p(rows), total, qo, qo_tok,
                                        qo_head, ko, ko_tok, ko_head, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(qo=None), EINVAL), (dict(ko=None), EINVAL),
    (dict(q=ODD), EINVAL), (dict(ko=ODD), EINVAL), (dict(qw=ODD), EINVAL), (dict(pos=ODD), EINVAL),
    (dict(dtype=3), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(dim=0), ESHAPE), (dict(dim=63), ESHAPE), (dict(dim=514), ESHAPE), (dict(heads=0), ESHAPE),
    (dict(k_heads=-1), ESHAPE), (dict(heads=1 << 20), ESHAPE), (dict(rope=_rope(freq=None)), EINVAL),
    (dict(rope=_rope(rot=66)), ESHAPE), (dict(rope=_rope(rot=-2)), ESHAPE), (dict(rope=_rope(rot=3)), ESHAPE),
    (dict(rope=_rope(amp=float("inf"))), EINVAL), (dict(rope=_rope(freq=ODD)), EINVAL),
    (dict(rows=None), EINVAL), (dict(rows=None, pos=A, total=-1), ESHAPE),
    (dict(rows=None, pos=A, total=(1 << 30) + 1), ESHAPE), (dict(total=9), ESHAPE),
    (dict(rows=_rows(cu=None)), EINVAL), (dict(rows=_rows(lens=ODD)), EINVAL),
    (dict(rows=_rows(seqs=65536)), ESHAPE), (dict(rows=_rows(max_rows=11)), ESHAPE),
    (dict(rows=_rows(seqs=-1)), EINVAL), (dict(q_head=63), ESHAPE), (dict(qo_head=32), ESHAPE),
    (dict(qo_tok=64), ESHAPE), (dict(qo_tok=0), ESHAPE), (dict(q_tok=1 << 50), ESHAPE),
    (dict(qo=A, qo_tok=512), EINVAL), (dict(qo=A, qo_head=80, qo_tok=512), EINVAL),
    (dict(rows=_rows(seqs=0), q=None), 0), (dict(rows=None, pos=A, total=0, q=None), 0),
    (dict(rows=_rows(total=0, max_rows=0), total=0, q=None), 0)])
def test_qk_refusals(kw, code):
    assert _qk(**kw) == code
    if code:
        _message("avae_qk_norm_rope")


# ------------------------------------------------------------------ cache

def _cache(k=A, v=B, ks=C, vs=D, n=8, heads=2, page=16, dim=64):
    return avae.avae_kv_q8(k, v, ks, vs, n, heads, page, dim)


def _write(k=A, k_tok=128, k_head=64, v=B, v_tok=128, v_head=64, dtype=0, weight=C, eps=1e-6,
           rope=DEFAULT, pos=None, cache=DEFAULT, rows=DEFAULT):
    rope, cache, rows = (d() if x is DEFAULT else x
                         for d, x in ((_rope, rope), (_cache, cache), (_rows, rows)))
    return avae.lib().avae_kv_write_rope_q8(k, k_tok, k_head, v, v_tok, v_head, dtype, weight, eps,
                                            _p(rope), pos, _p(cache), _p(rows), None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(v=ODD), EINVAL), (dict(weight=ODD), EINVAL),
    (dict(pos=ODD), EINVAL), (dict(dtype=-1), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(cache=None), EINVAL), (dict(cache=_cache(ks=None)), EINVAL), (dict(cache=_cache(page=24)), ESHAPE),
    (dict(cache=_cache(dim=96)), ESHAPE), (dict(rows=None), EINVAL), (dict(rows=_rows(table=None)), EINVAL),
    (dict(rows=_rows(ld=3)), ESHAPE), (dict(rope=_rope(rot=128)), ESHAPE), (dict(rope=_rope(rot=5)), ESHAPE),
    (dict(rope=_rope(freq=None)), EINVAL), (dict(k_head=63), ESHAPE), (dict(v_tok=-1), ESHAPE),
    (dict(rows=_rows(seqs=0), k=None), 0), (dict(rows=_rows(max_rows=0), k=None), 0)])
def test_write_refusals(kw, code):
    assert _write(**kw) == code
    if code:
        _message("avae_kv_write_rope_q8")


# ------------------------------------------------------------------ attention

def _rules(cap=0.0, slopes=None, prefix=None, max_prefix=0, tree=None, ld=1, words=1):
    return avae.avae_attn_rules(cap, slopes, prefix, max_prefix, tree, ld, words)


def _attn(q=A, tok=256, head=64, heads=4, dtype=1, cache=DEFAULT, rows=DEFAULT, first=None, max_len=64,
          scale=0.125, causal=1, window=0, rules=DEFAULT, out=B, lse=None, ws=A, ws_bytes=1 << 40):
    cache, rows, rules = (d() if x is DEFAULT else x
                          for d, x in ((_cache, cache), (_rows, rows), (_rules, rules)))
    return avae.lib().avae_attn_rules_q8(q, tok, head, heads, dtype, _p(cache), _p(rows), first,
                                         max_len, scale, causal, window, _p(rules), out, lse, ws,
                                         ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rules=None), EINVAL), (dict(rules=_rules(cap=-1.0)), EINVAL),
    (dict(rules=_rules(cap=float("nan"))), EINVAL), (dict(rules=_rules(cap=float("inf"))), EINVAL),
    (dict(rules=_rules(cap=1e-38)), EINVAL), (dict(rules=_rules(slopes=ODD)), EINVAL),
    (dict(rules=_rules(prefix=ODD)), EINVAL), (dict(rules=_rules(tree=ODD)), EINVAL),
    (dict(rules=_rules(prefix=A), causal=0), EINVAL), (dict(rules=_rules(prefix=A, max_prefix=-1)), EINVAL),
    (dict(rules=_rules(tree=A), window=5), EINVAL), (dict(rules=_rules(tree=A), causal=0), EINVAL),
    (dict(rules=_rules(tree=A, slopes=B)), EINVAL), (dict(rules=_rules(tree=A, prefix=B)), EINVAL),
    (dict(rules=_rules(tree=A, words=0)), ESHAPE), (dict(rules=_rules(tree=A, words=129, ld=129)), ESHAPE),
    (dict(rules=_rules(tree=A, words=2, ld=1)), ESHAPE),
    (dict(rules=_rules(tree=A), rows=_rows(total=40, max_rows=33)), ESHAPE),
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(heads=3), ESHAPE), (dict(heads=0), ESHAPE),
    (dict(dtype=7), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(max_len=65), ESHAPE),
    (dict(max_len=-1), EINVAL), (dict(window=4, causal=0), EINVAL), (dict(out=ODD), EINVAL),
    (dict(lse=ODD), EINVAL), (dict(first=ODD), EINVAL), (dict(cache=_cache(dim=32)), ESHAPE),
    (dict(rows=_rows(cu=None)), EINVAL), (dict(head=10), ESHAPE),
    (dict(rows=_rows(seqs=0), q=None), 0), (dict(rows=_rows(total=0, max_rows=0), q=None), 0)])
def test_attention_refusals(kw, code):
    assert _attn(**kw) == code
    if code:
        _message("avae_attn_rules_q8")


def test_attention_workspace():
    """A split call without room is refused; a prefix beside a window makes
    more keys of it, a prefix alone does not."""
    L = avae.lib()
    cache, rows = _cache(n=4096), _rows(cols=4096, ld=4096, seqs=1, total=1, max_rows=1)

    def need(window, rules):
        return L.avae_attn_rules_q8_workspace_bytes(_p(cache), _p(rows), 4, 1, 50000, window, _p(rules))

    assert need(0, _rules()) == need(0, _rules(prefix=A, max_prefix=20000)) > 0
    assert need(100, _rules(prefix=A, max_prefix=20000)) > need(100, _rules(prefix=A)) >= 0
    assert need(0, _rules()) == L.avae_attn_q8_workspace_bytes(_p(cache), _p(rows), 4, 1, 50000, 0)
    assert _attn(cache=cache, rows=rows, max_len=50000, ws=None, ws_bytes=0) == EWORKSPACE
    assert _attn(cache=cache, rows=rows, max_len=50000, ws_bytes=need(0, _rules()) - 1) == EWORKSPACE
    assert _attn(cache=cache, rows=rows, max_len=50000, ws=ODD) == EWORKSPACE


# ------------------------------------------------------------------ masks

def _mask(parents=A, rows=DEFAULT, words=1, mask=B, ld=1, pos=C):
    rows = _rows(table=None, ld=0, cols=0) if rows is DEFAULT else rows
    return avae.lib().avae_tree_mask(parents, _p(rows), words, mask, ld, pos, None)


@pytest.mark.parametrize("kw,code", [
    (dict(parents=None), EINVAL), (dict(mask=None), EINVAL), (dict(parents=ODD), EINVAL), (dict(pos=ODD), EINVAL),
    (dict(rows=None), EINVAL), (dict(rows=_rows(cu=None)), EINVAL), (dict(words=-1), ESHAPE),
    (dict(words=129), ESHAPE), (dict(words=0), ESHAPE), (dict(words=2), ESHAPE),
    (dict(rows=_rows(total=40, max_rows=33)), ESHAPE), (dict(rows=_rows(max_rows=-1)), EINVAL),
    (dict(rows=_rows(seqs=0), mask=None), 0), (dict(rows=_rows(max_rows=0), words=0, mask=None), 0)])
def test_mask_refusals(kw, code):
    assert _mask(**kw) == code
    if code:
        _message("avae_tree_mask")


# ------------------------------------------------------------------ the binding's own checks

def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch
    with pytest.raises(ValueError):
        avae.Rope(torch.ones(32))
    with pytest.raises(ValueError):
        avae.qk_norm_rope(torch.ones(2, 3, 64), None, None, positions=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        avae.qk_norm_rope(torch.ones(2, 64), None, None)
    with pytest.raises(ValueError):
        avae.tree_mask(torch.zeros(3, 2, dtype=torch.int32), None, torch.zeros(1, dtype=torch.int32))
