"""Refusals of the 8-bit serving operators: every bad argument is a code and
a message before anything touches a device (no GPU is needed)."""
import ctypes

import pytest

from bigvgan_waveform_decoder_amd import avae

EINVAL, ESHAPE, EWORKSPACE = -1, -2, -3
A, B, C, D = (ctypes.c_void_p(v) for v in (0x10000, 0x20000, 0x30000, 0x40000))
ODD = ctypes.c_void_p(0x10001)


def _norm(x=A, ldx=64, res=None, ldr=64, w=B, M=2, C_=64, dtype=1, eps=1e-6, total=None, lds=64, q=C,
          ldq=64, scale=D):
    return avae.lib().avae_rms_norm_q8(x, ldx, res, ldr, w, M, C_, dtype, eps, total, lds, q, ldq,
                                       scale, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(q=None), EINVAL), (dict(scale=None), EINVAL),
    (dict(M=-1), EINVAL), (dict(C_=0), EINVAL), (dict(dtype=3), EINVAL), (dict(dtype=-1), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(res=B), EINVAL), (dict(total=B), EINVAL), (dict(res=B, total=A), EINVAL),
    (dict(res=B, total=B), EINVAL), (dict(x=ODD), EINVAL), (dict(w=ODD), EINVAL),
    (dict(ldx=63), ESHAPE), (dict(ldq=63), ESHAPE), (dict(ldx=1 << 50), ESHAPE),
    (dict(res=B, total=C, ldr=10), ESHAPE), (dict(res=B, total=C, lds=10), ESHAPE),
    (dict(M=0, x=None, q=None), 0)])
def test_norm_refusals(kw, code):
    assert _norm(**kw) == code
    if code:
        assert avae.lib().avae_last_error().startswith(b"avae_rms_norm_q8: ")


def test_rows_refusals():
    L = avae.lib()
    assert L.avae_quant_q8(None, 8, 2, 8, 0, A, 8, B, None) == EINVAL
    assert L.avae_quant_q8(A, 7, 2, 8, 0, B, 8, C, None) == ESHAPE
    assert L.avae_quant_q8(A, 8, 2, 8, 7, B, 8, C, None) == EINVAL
    assert L.avae_quant_q8(None, 8, 0, 8, 0, None, 8, None, None) == 0
    assert L.avae_dequant_q8(A, 8, None, 2, 8, 0, C, 8, None) == EINVAL
    assert L.avae_dequant_q8(A, 8, B, 2, 8, 0, C, 7, None) == ESHAPE
    assert L.avae_dequant_q8(A, 8, B, 2, 8, 0, ODD, 8, None) == EINVAL
    assert L.avae_dequant_q8(A, 8, B, -2, 8, 0, C, 8, None) == EINVAL


def _linear(a=A, lda=64, sa=B, w=C, ldw=64, sw=D, bias=None, M=2, N=3, K=64, act=0, dtype=0, y=B,
            ldy=3, ws=A, ws_bytes=1 << 40):
    return avae.lib().avae_linear_q8(a, lda, sa, w, ldw, sw, bias, M, N, K, act, dtype, y, ldy, ws,
                                     ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), EINVAL), (dict(sa=None), EINVAL), (dict(w=None), EINVAL), (dict(sw=None), EINVAL),
    (dict(y=None), EINVAL), (dict(M=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL),
    (dict(act=2), EINVAL), (dict(dtype=9), EINVAL), (dict(bias=ODD), EINVAL), (dict(y=ODD), EINVAL),
    (dict(K=131072, lda=131072, ldw=131072), ESHAPE), (dict(lda=63), ESHAPE), (dict(ldw=63), ESHAPE),
    (dict(ldy=2), ESHAPE), (dict(M=1 << 22), ESHAPE), (dict(M=0, a=None), 0)])
def test_linear_refusals(kw, code):
    assert _linear(**kw) == code
    if code:
        assert avae.lib().avae_last_error().startswith(b"avae_linear_q8: ")


def test_linear_workspace():
    L = avae.lib()
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 131072)):
        assert L.avae_linear_q8_workspace_bytes(*bad) == 0
    for M, N, K in ((1, 64, 131071), (2, 128, 65536), (64, 64, 8192)):
        need = L.avae_linear_q8_workspace_bytes(M, N, K)
        if need:
            assert _linear(M=M, N=N, K=K, lda=K, ldw=K, ldy=N, ws_bytes=need - 1) == EWORKSPACE
            assert _linear(M=M, N=N, K=K, lda=K, ldw=K, ldy=N, ws=None) == EWORKSPACE
            assert _linear(M=M, N=N, K=K, lda=K, ldw=K, ldy=N, ws=ODD) == EWORKSPACE


def _cache(**kw):
    f = dict(k=0x10000, v=0x20000, k_scale=0x30000, v_scale=0x40000, n_pages=8, heads=2, page=16,
             dim=64)
    f.update(kw)
    return avae.avae_kv_q8(*(f[n] for n, _ in avae.avae_kv_q8._fields_))


def _rows(**kw):
    f = dict(cu=0x50000, lens=0x60000, table=0x70000, table_ld=4, table_cols=4, seqs=2, total=5,
             max_rows=3)
    f.update(kw)
    return avae.avae_ragged(*(f[n] for n, _ in avae.avae_ragged._fields_))


BAD_CACHE = [(dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(k_scale=None), EINVAL),
             (dict(v_scale=None), EINVAL), (dict(n_pages=0), EINVAL), (dict(heads=0), EINVAL),
             (dict(heads=5000), ESHAPE), (dict(page=24), ESHAPE), (dict(page=8), ESHAPE),
             (dict(page=512), ESHAPE), (dict(dim=96), ESHAPE), (dict(dim=32), ESHAPE),
             (dict(k=0x10008), EINVAL), (dict(v=0x20001), EINVAL), (dict(k_scale=0x30002), EINVAL)]
BAD_ROWS = [(dict(cu=None), EINVAL), (dict(lens=None), EINVAL), (dict(table=None), EINVAL),
            (dict(seqs=-1), EINVAL), (dict(total=-1), EINVAL), (dict(max_rows=-1), EINVAL),
            (dict(max_rows=6), ESHAPE), (dict(table_cols=0), ESHAPE), (dict(table_ld=3), ESHAPE),
            (dict(seqs=70000), ESHAPE), (dict(table_cols=1 << 28, table_ld=1 << 28), ESHAPE),
            (dict(lens=0x60002), EINVAL), (dict(total=0, max_rows=0), 0),
            (dict(seqs=0, cu=None, lens=None, table=None), 0)]


@pytest.mark.parametrize("cache,rows,code", [(k, {}, c) for k, c in BAD_CACHE]
                         + [({}, k, c) for k, c in BAD_ROWS])
def test_cache_and_sequence_refusals(cache, rows, code):
    L = avae.lib()
    c, r = _cache(**cache), _rows(**rows)
    pc, pr = ctypes.byref(c), ctypes.byref(r)
    assert L.avae_kv_write_q8(A, 128, 64, B, 128, 64, 1, pc, pr, None) == code
    assert L.avae_kv_read_q8(pc, pr, 0, A, B, None) == code
    assert L.avae_attn_q8(A, 256, 64, 4, 1, pc, pr, None, 60, 0.1, 1, 0, B, None, C, 1 << 40,
                          None) == code


def test_write_and_read_refusals():
    L = avae.lib()
    c, r = _cache(), _rows()
    pc, pr = ctypes.byref(c), ctypes.byref(r)
    assert L.avae_kv_write_q8(None, 128, 64, B, 128, 64, 1, pc, pr, None) == EINVAL
    assert L.avae_kv_write_q8(A, 128, 64, None, 128, 64, 1, pc, pr, None) == EINVAL
    assert L.avae_kv_write_q8(A, 128, 64, B, 128, 64, 4, pc, pr, None) == EINVAL
    assert L.avae_kv_write_q8(ODD, 128, 64, B, 128, 64, 1, pc, pr, None) == EINVAL
    assert L.avae_kv_write_q8(A, 128, 32, B, 128, 64, 1, pc, pr, None) == ESHAPE
    assert L.avae_kv_write_q8(A, 128, 64, B, -1, 64, 1, pc, pr, None) == ESHAPE
    assert L.avae_kv_write_q8(A, 128, 64, B, 128, 64, 1, None, pr, None) == EINVAL
    assert L.avae_kv_write_q8(A, 128, 64, B, 128, 64, 1, pc, None, None) == EINVAL
    assert L.avae_kv_read_q8(pc, pr, 0, None, B, None) == EINVAL
    assert L.avae_kv_read_q8(pc, pr, 0, A, ODD, None) == EINVAL


def _attn(q=A, tok=256, head=64, heads=4, dtype=1, first=None, max_len=60, scale=0.1, causal=1,
          window=0, out=B, lse=None, ws=C, ws_bytes=1 << 40, cache=None, rows=None):
    c, r = cache or _cache(), rows or _rows()
    return avae.lib().avae_attn_q8(q, tok, head, heads, dtype, ctypes.byref(c), ctypes.byref(r),
                                   first, max_len, scale, causal, window, out, lse, ws, ws_bytes,
                                   None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(heads=3), ESHAPE), (dict(heads=0), ESHAPE),
    (dict(heads=4096), ESHAPE), (dict(dtype=5), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(max_len=-1), EINVAL), (dict(max_len=65), ESHAPE),
    (dict(window=-1), EINVAL), (dict(window=4, causal=0), EINVAL), (dict(head=32), ESHAPE),
    (dict(tok=-5), ESHAPE), (dict(q=ODD), EINVAL), (dict(lse=ODD), EINVAL), (dict(first=ODD), EINVAL)])
def test_attention_refusals(kw, code):
    assert _attn(**kw) == code
    assert avae.lib().avae_last_error().startswith(b"avae_attn_q8: ")


def test_attention_workspace():
    L = avae.lib()
    c = _cache(n_pages=1000)
    r = _rows(table_cols=500, table_ld=500, seqs=1, total=1, max_rows=1)
    pc, pr = ctypes.byref(c), ctypes.byref(r)
    assert L.avae_attn_q8_workspace_bytes(None, pr, 4, 1, 100, 0) == 0
    assert L.avae_attn_q8_workspace_bytes(pc, pr, 3, 1, 100, 0) == 0
    need = L.avae_attn_q8_workspace_bytes(pc, pr, 4, 1, 8000, 0)
    if need:
        for kw in (dict(ws_bytes=need - 1), dict(ws=None), dict(ws=ODD)):
            assert _attn(cache=c, rows=r, max_len=8000, **kw) == EWORKSPACE


def test_binding_checks_tensors():
    """What the binding refuses before the library is asked."""
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 8))
    with pytest.raises(ValueError, match="device tensor"):
        avae.quant_q8(x)
    with pytest.raises(ValueError, match="dtype"):
        avae.quant_q8(x.double())
    with pytest.raises(ValueError, match="device tensor"):
        avae.KvCacheQ8(*(torch.zeros((1, 1, 16, 64), dtype=torch.int8) for _ in range(2)),
                       *(torch.zeros((1, 1)) for _ in range(2)))


def test_linear_columns_of_one_launch():
    assert _linear(N=1 << 28, ldy=1 << 28) == ESHAPE


def test_more_work_than_a_launch_takes():
    """Bounds of the rows that are far from the truth are refused by name."""
    L = avae.lib()
    many = dict(seqs=60000, total=1 << 20, max_rows=1 << 20)
    assert _attn(rows=_rows(**many)) == ESHAPE
    assert b"workgroups" in L.avae_last_error() and b"split the call" in L.avae_last_error()
    # (few rows over split keys, in packed rows far longer than they are)
    assert _attn(cache=_cache(n_pages=1000), max_len=40000, ws_bytes=1 << 62,
                 rows=_rows(table_cols=2500, table_ld=2500, seqs=1, total=1 << 25, max_rows=1)) == ESHAPE
    assert b"workgroups" in L.avae_last_error()
    c, r = _cache(), _rows(table_cols=1 << 25, table_ld=1 << 25, total=1 << 30, max_rows=1 << 29)
    assert L.avae_kv_write_q8(A, 128, 64, B, 128, 64, 1, ctypes.byref(c), ctypes.byref(r), None) == ESHAPE
    assert b"2^24 pages" in L.avae_last_error()


@pytest.mark.parametrize("M,N,K", [(1000, 1000, 77), (64, 10000, 1001), (6000, 6143, 1535)])
def test_linear_workspace_of_odd_rows(M, N, K):
    """Products large enough for tiles with rows of odd length do need one."""
    need = avae.lib().avae_linear_q8_workspace_bytes(M, N, K)
    assert need >= (M + N) * K
    kw = dict(M=M, N=N, K=K, lda=K, ldw=K, ldy=N)
    for bad in (dict(ws_bytes=need - 1), dict(ws=None), dict(ws=ODD), dict(ws_bytes=0)):
        assert _linear(**kw, **bad) == EWORKSPACE


def test_attention_workspace_of_split_keys():
    c = _cache(n_pages=1000)
    rows = dict(table_cols=500, table_ld=500, seqs=1, total=1, max_rows=1)
    need = avae.lib().avae_attn_q8_workspace_bytes(ctypes.byref(c), ctypes.byref(_rows(**rows)), 4, 1,
                                                   8000, 0)
    assert need > 0
    for bad in (dict(ws_bytes=need - 1), dict(ws=None), dict(ws=ODD), dict(ws_bytes=0)):
        assert _attn(cache=c, rows=_rows(**rows), max_len=8000, **bad) == EWORKSPACE
