"""Thin ctypes binding over libavae.so (see include/avae.h).

Argument marshalling only: every step of the decoder runs in the library's
HIP kernels.  PyTorch provides device memory (``tensor.data_ptr()``) and the
stream (``torch.cuda.current_stream().cuda_stream``).  There is no fallback:
if the library is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, List, Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# AVAE_LIB_PATH selects another build of the same library (the host-sanitized
# check build); a missing file raises like a missing default.
LIB_PATH = os.environ.get("AVAE_LIB_PATH") or os.path.join(_HERE, "libavae.so")

AVAE_FILTER_LEN = 12
AVAE_MAX_STAGES = 8
AVAE_MAX_KERNELS = 4
AVAE_MAX_DIL = 4
FINAL = {"none": 0, "tanh": 1, "clamp": 2}

c_int, c_float, c_double, c_size_t, c_void_p = (ctypes.c_int, ctypes.c_float, ctypes.c_double,
                                                ctypes.c_size_t, ctypes.c_void_p)
P = c_void_p


class AvaeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libavae error {code}: {msg}")
        self.code = code


class avae_config(ctypes.Structure):
    _fields_ = [
        ("c_in", c_int), ("dec_in_ch", c_int), ("has_latent_affine", c_int),
        ("k_pre", c_int), ("k_post", c_int), ("n_stages", c_int),
        ("ch", c_int * (AVAE_MAX_STAGES + 1)),
        ("rates", c_int * AVAE_MAX_STAGES), ("up_k", c_int * AVAE_MAX_STAGES),
        ("n_kernels", c_int), ("rb_k", c_int * AVAE_MAX_KERNELS), ("n_dil", c_int),
        ("rb_d", (c_int * AVAE_MAX_DIL) * AVAE_MAX_KERNELS), ("final_act", c_int),
    ]


_W3 = ((P * AVAE_MAX_DIL) * AVAE_MAX_KERNELS) * AVAE_MAX_STAGES
_A3 = ((P * (2 * AVAE_MAX_DIL)) * AVAE_MAX_KERNELS) * AVAE_MAX_STAGES


class avae_weights(ctypes.Structure):
    _fields_ = [
        ("latent_mean", P), ("latent_std", P), ("dec_in_w", P), ("dec_in_b", P),
        ("conv_pre_w", P), ("conv_pre_b", P),
        ("up_w", P * AVAE_MAX_STAGES), ("up_b", P * AVAE_MAX_STAGES),
        ("w1", _W3), ("b1", _W3), ("w2", _W3), ("b2", _W3),
        ("act_la", _A3), ("act_lb", _A3),
        ("post_la", P), ("post_lb", P), ("conv_post_w", P), ("conv_post_b", P),
    ]


class avae_dav_config(ctypes.Structure):
    _fields_ = [
        ("c_side", c_int), ("dec_in_ch", c_int), ("k_pre", c_int), ("k_post", c_int),
        ("n_stages", c_int), ("ch", c_int * (AVAE_MAX_STAGES + 1)),
        ("strides", c_int * AVAE_MAX_STAGES), ("up_k", c_int * AVAE_MAX_STAGES),
        ("unit_k", c_int), ("n_units", c_int), ("unit_dil", c_int * AVAE_MAX_DIL),
    ]


_U2 = (P * AVAE_MAX_DIL) * AVAE_MAX_STAGES


class avae_dav_weights(ctypes.Structure):
    _fields_ = [
        ("dec_in_w", P), ("dec_in_b", P), ("conv_pre_w", P), ("conv_pre_b", P),
        ("stage_alpha", P * AVAE_MAX_STAGES), ("up_w", P * AVAE_MAX_STAGES),
        ("up_b", P * AVAE_MAX_STAGES),
        ("a1", _U2), ("w1", _U2), ("b1", _U2), ("a2", _U2), ("w2", _U2), ("b2", _U2),
        ("post_alpha", P), ("conv_post_w", P), ("conv_post_b", P),
    ]


class avae_bwe_config(ctypes.Structure):
    _fields_ = [("gen", avae_config), ("filter_len", c_int), ("hop", c_int), ("n_freqs", c_int),
                ("n_mels", c_int), ("ratio", c_int)]


class avae_bwe_weights(ctypes.Structure):
    _fields_ = [("gen", avae_weights), ("forward_basis", P), ("mel_basis", P)]


class avae_kv_q8(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P),
                ("n_pages", c_int), ("heads", c_int), ("page", c_int), ("dim", c_int)]


class avae_ragged(ctypes.Structure):
    _fields_ = [("cu", P), ("lens", P), ("table", P), ("table_ld", ctypes.c_longlong),
                ("table_cols", c_int), ("seqs", c_int), ("total", c_int), ("max_rows", c_int)]


class avae_rope(ctypes.Structure):
    _fields_ = [("freq", P), ("rot", c_int), ("interleaved", c_int), ("amp", c_float)]


class avae_attn_rules(ctypes.Structure):
    _fields_ = [("cap", c_float), ("slopes", P), ("prefix", P), ("max_prefix", c_int),
                ("tree", P), ("tree_ld", ctypes.c_longlong), ("tree_words", c_int)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                           "(python -m bigvgan_waveform_decoder_amd.build)")
    L = ctypes.CDLL(LIB_PATH)
    L.avae_last_error.restype = ctypes.c_char_p
    L.avae_last_error.argtypes = []
    L.avae_version.restype = c_int
    L.avae_kaiser_sinc.restype = c_int
    L.avae_kaiser_sinc.argtypes = [c_double, c_double, c_int, P]
    L.avae_act1d.restype = c_int
    L.avae_act1d.argtypes = [P, P, c_int, c_int, c_int, P, P, P, P, P]
    L.avae_conv1d.restype = c_int
    L.avae_conv1d.argtypes = [P, P, c_int, c_int, c_int, c_int, P, P, c_int, c_int, c_int, P, P]
    L.avae_conv1d_fft_weight_floats.restype = c_size_t
    L.avae_conv1d_fft_weight_floats.argtypes = [c_int, c_int]
    L.avae_conv1d_fft_pack.restype = c_int
    L.avae_conv1d_fft_pack.argtypes = [P, P, c_int, c_int, c_int, c_int, P]
    L.avae_conv1d_fft_workspace_bytes.restype = c_size_t
    L.avae_conv1d_fft_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int, c_int]
    L.avae_conv1d_fft.restype = c_int
    L.avae_conv1d_fft.argtypes = [P, P, c_int, c_int, c_int, c_int, P, P, c_int, c_int, P, P,
                                  c_size_t, P]
    L.avae_act_conv1d_fft.restype = c_int
    L.avae_act_conv1d_fft.argtypes = [P, P, c_int, c_int, c_int, c_int, P, P, P, P, c_int, c_int,
                                      P, P, c_size_t, P]
    L.avae_convtr1d.restype = c_int
    L.avae_convtr1d.argtypes = [P, P, c_int, c_int, c_int, c_int, P, P, c_int, c_int, c_int, P]
    L.avae_amp_block_workspace_bytes.restype = c_size_t
    L.avae_amp_block_workspace_bytes.argtypes = [c_int, c_int, c_int]
    L.avae_amp_block_fft_workspace_bytes.restype = c_size_t
    L.avae_amp_block_fft_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int, c_int, P]
    L.avae_amp_block.restype = c_int
    L.avae_amp_block.argtypes = [P, P, c_int, c_int, c_int, c_int, c_int, P, P, P, P, P, P, P,
                                 c_float, c_int, P, c_size_t, P]
    L.avae_amp_block_static_max_bytes.restype = c_size_t
    L.avae_amp_block_static_max_bytes.argtypes = []
    L.avae_amp_block_static.restype = c_int
    L.avae_amp_block_static.argtypes = [P, P, c_int, c_int, c_int, c_int, c_int, P, P, P, P, P,
                                        P, P, c_float, c_int, P]
    L.avae_decoder_create.restype = c_int
    L.avae_decoder_create.argtypes = [ctypes.POINTER(avae_config), ctypes.POINTER(avae_weights),
                                      ctypes.POINTER(P)]
    L.avae_decoder_destroy.restype = None
    L.avae_decoder_destroy.argtypes = [P]
    L.avae_decoder_output_length.restype = c_int
    L.avae_decoder_output_length.argtypes = [P, c_int, ctypes.POINTER(c_int)]
    L.avae_decoder_workspace_bytes.restype = c_size_t
    L.avae_decoder_workspace_bytes.argtypes = [P, c_int, c_int]
    L.avae_decoder_set_concurrent.restype = c_int
    L.avae_decoder_set_concurrent.argtypes = [P, c_int]
    L.avae_probe_mfma.restype = c_int
    L.avae_probe_mfma.argtypes = [c_int, c_int, c_int, P, P]
    L.avae_probe_copy.restype = c_int
    L.avae_probe_copy.argtypes = [P, P, ctypes.c_longlong, P]
    L.avae_bigvgan_decode.restype = c_int
    L.avae_bigvgan_decode.argtypes = [P, P, c_int, c_int, P, P, c_size_t, P]
    L.avae_bigvgan_decode_traced.restype = c_int
    L.avae_bigvgan_decode_traced.argtypes = [P, P, c_int, c_int, P, P, c_size_t, P, P]
    L.avae_mel_stft.restype = c_int
    L.avae_mel_stft.argtypes = [P, P, c_int, c_int, P, c_int, c_int, c_int, P, c_int, P]
    L.avae_hann_sinc_upsample.restype = c_int
    L.avae_hann_sinc_upsample.argtypes = [P, P, c_int, c_int, c_int, P]
    L.avae_bwe_create.restype = c_int
    L.avae_bwe_create.argtypes = [P, P, P]
    L.avae_bwe_destroy.restype = None
    L.avae_bwe_destroy.argtypes = [P]
    L.avae_bwe_workspace_bytes.restype = c_size_t
    L.avae_bwe_workspace_bytes.argtypes = [P, c_int, c_int]
    L.avae_bwe_decode.restype = c_int
    L.avae_bwe_decode.argtypes = [P, P, c_int, c_int, P, P, c_size_t, P]
    L.avae_bwe_decode_traced.restype = c_int
    L.avae_bwe_decode_traced.argtypes = [P, P, c_int, c_int, P, P, c_size_t, P, P, P]
    L.avae_snake.restype = c_int
    L.avae_snake.argtypes = [P, P, c_int, c_int, c_int, P, P]
    L.avae_dav_create.restype = c_int
    L.avae_dav_create.argtypes = [P, P, P]
    L.avae_dav_destroy.restype = None
    L.avae_dav_destroy.argtypes = [P]
    L.avae_dav_output_length.restype = c_int
    L.avae_dav_output_length.argtypes = [P, c_int, ctypes.POINTER(c_int)]
    L.avae_dav_workspace_bytes.restype = c_size_t
    L.avae_dav_workspace_bytes.argtypes = [P, c_int, c_int]
    L.avae_dav_decode.restype = c_int
    L.avae_dav_decode.argtypes = [P, P, c_int, c_int, P, P, c_size_t, P]
    L.avae_dav_decode_traced.restype = c_int
    L.avae_dav_decode_traced.argtypes = [P, P, c_int, c_int, P, P, c_size_t, P, P]
    L.avae_decoder_reach_frames.restype = c_int
    L.avae_decoder_reach_frames.argtypes = [P, ctypes.POINTER(c_int)]
    L.avae_decoder_streaming_workspace_bytes.restype = c_size_t
    L.avae_decoder_streaming_workspace_bytes.argtypes = [P, c_int, c_int, c_int]
    L.avae_bigvgan_decode_streaming.restype = c_int
    L.avae_bigvgan_decode_streaming.argtypes = [P, P, c_int, c_int, P, c_int, c_int, P, c_size_t, P]
    LL = ctypes.c_longlong
    L.avae_rms_norm_q8.restype = c_int
    L.avae_rms_norm_q8.argtypes = [P, LL, P, LL, P, c_int, c_int, c_int, c_float, P, LL, P, LL, P,
                                   P]
    L.avae_quant_q8.restype = c_int
    L.avae_quant_q8.argtypes = [P, LL, c_int, c_int, c_int, P, LL, P, P]
    L.avae_dequant_q8.restype = c_int
    L.avae_dequant_q8.argtypes = [P, LL, P, c_int, c_int, c_int, P, LL, P]
    L.avae_linear_q8_workspace_bytes.restype = c_size_t
    L.avae_linear_q8_workspace_bytes.argtypes = [c_int, c_int, c_int]
    L.avae_linear_q8.restype = c_int
    L.avae_linear_q8.argtypes = [P, LL, P, P, LL, P, P, c_int, c_int, c_int, c_int, c_int, P, LL,
                                 P, c_size_t, P]
    L.avae_kv_write_q8.restype = c_int
    L.avae_kv_write_q8.argtypes = [P, LL, LL, P, LL, LL, c_int, P, P, P]
    L.avae_kv_read_q8.restype = c_int
    L.avae_kv_read_q8.argtypes = [P, P, c_int, P, P, P]
    L.avae_attn_q8_workspace_bytes.restype = c_size_t
    L.avae_attn_q8_workspace_bytes.argtypes = [P, P, c_int, c_int, c_int, c_int]
    L.avae_attn_q8.restype = c_int
    L.avae_attn_q8.argtypes = [P, LL, LL, c_int, c_int, P, P, P, c_int, c_float, c_int, c_int, P,
                               P, P, c_size_t, P]
    L.avae_rope_freq.restype = c_int
    L.avae_rope_freq.argtypes = [c_int, c_double, c_int, c_double, c_double, c_double, c_double, P,
                                 P]
    L.avae_qk_norm_rope.restype = c_int
    L.avae_qk_norm_rope.argtypes = [P, LL, LL, c_int, P, P, LL, LL, c_int, P, c_int, c_int,
                                    c_float, P, P, P, c_int, P, LL, LL, P, LL, LL, P]
    L.avae_kv_write_rope_q8.restype = c_int
    L.avae_kv_write_rope_q8.argtypes = [P, LL, LL, P, LL, LL, c_int, P, c_float, P, P, P, P, P]
    L.avae_attn_rules_q8_workspace_bytes.restype = c_size_t
    L.avae_attn_rules_q8_workspace_bytes.argtypes = [P, P, c_int, c_int, c_int, c_int, P]
    L.avae_attn_rules_q8.restype = c_int
    L.avae_attn_rules_q8.argtypes = [P, LL, LL, c_int, c_int, P, P, P, c_int, c_float, c_int,
                                     c_int, P, P, P, P, c_size_t, P]
    L.avae_tree_mask.restype = c_int
    L.avae_tree_mask.argtypes = [P, P, c_int, P, LL, P, P]
    L.avae_profile_begin.restype = c_int
    L.avae_profile_begin.argtypes = [c_int]
    L.avae_profile_end.restype = c_int
    L.avae_profile_end.argtypes = []
    L.avae_profile_count.restype = c_int
    L.avae_profile_count.argtypes = []
    L.avae_profile_entry.restype = c_int
    L.avae_profile_entry.argtypes = [c_int, ctypes.c_char_p, c_int,
                                     ctypes.POINTER(ctypes.c_longlong),
                                     ctypes.POINTER(c_double), ctypes.POINTER(c_double),
                                     ctypes.POINTER(c_double)]
    L.avae_profile_phases.restype = c_int
    L.avae_profile_phases.argtypes = [ctypes.POINTER(c_double)]
    _lib = L
    return L


def _check(rc: int):
    if rc != 0:
        raise AvaeError(rc, lib().avae_last_error().decode())


# ------------------------------------------------------------------ helpers

def _torch():
    import torch
    return torch


def _dev(t, name: str, shape: Optional[Sequence[int]] = None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if t.dtype != torch.float32:
        raise ValueError(f"{name}: must be float32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _opt(t, name, shape=None):
    return None if t is None else _dev(t, name, shape)


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _host_taps(taps):
    if taps is None:
        return None, None
    a = np.ascontiguousarray(np.asarray(taps, dtype=np.float32))
    if a.shape != (AVAE_FILTER_LEN,):
        raise ValueError(f"taps must have {AVAE_FILTER_LEN} entries")
    return a, a.ctypes.data


# ------------------------------------------------------------------ entry points

def version() -> int:
    return lib().avae_version()


PHASES = ("dec_in", "conv_pre", "upsamples", "resblocks", "act_post", "conv_post")


def profile_begin(max_launches: int):
    """Open a profiled region (avae_profile_begin)."""
    _check(lib().avae_profile_begin(int(max_launches)))


def profile_end():
    """Close the region; returns (per-kernel dict, per-phase ms dict).
    Per kernel: launches, total_ms, flops, bytes (algorithmic, summed)."""
    L = lib()
    _check(L.avae_profile_end())
    out = {}
    for i in range(L.avae_profile_count()):
        name = ctypes.create_string_buffer(256)
        n = ctypes.c_longlong()
        ms, fl, by = c_double(), c_double(), c_double()
        _check(L.avae_profile_entry(i, name, 256, ctypes.byref(n), ctypes.byref(ms),
                                    ctypes.byref(fl), ctypes.byref(by)))
        out[name.value.decode()] = {"launches": n.value, "total_ms": ms.value,
                                    "flops": fl.value, "bytes": by.value}
    ph = (c_double * 6)()
    _check(L.avae_profile_phases(ph))
    return out, dict(zip(PHASES, list(ph)))


def kaiser_sinc(cutoff: float = 0.25, half_width: float = 0.3, taps: int = 12) -> np.ndarray:
    out = np.zeros(max(int(taps), 1), dtype=np.float32)
    _check(lib().avae_kaiser_sinc(cutoff, half_width, int(taps), out.ctypes.data))
    return out


def act1d(x, log_alpha, log_beta, up_taps=None, down_taps=None, out=None, stream=None):
    """avae_act1d: [B, C, T] -> [B, C, T]."""
    torch = _torch()
    B, C, T = x.shape
    px = _dev(x, "x")
    if out is None:
        out = torch.empty_like(x)
    py = _dev(out, "out", (B, C, T))
    ua, up = _host_taps(up_taps)
    da, dp = _host_taps(down_taps)
    _check(lib().avae_act1d(px, py, B, C, T, _dev(log_alpha, "log_alpha", (C,)),
                            _dev(log_beta, "log_beta", (C,)), up, dp, _stream(stream)))
    return out


def conv1d(x, w, bias=None, dilation: int = 1, pad: Optional[int] = None, residual=None,
           out=None, stream=None):
    """avae_conv1d; pad defaults to the 'same' padding (K*d - d)/2."""
    torch = _torch()
    B, Cin, T = x.shape
    Cout, Cin_w, K = w.shape
    if Cin_w != Cin:
        raise ValueError(f"weight has {Cin_w} input channels, x has {Cin}")
    if pad is None:
        pad = (K * dilation - dilation) // 2
    Tout = T + 2 * pad - dilation * (K - 1)
    if out is None:
        out = torch.empty((B, Cout, max(Tout, 0)), device=x.device, dtype=torch.float32)
    _check(lib().avae_conv1d(_dev(x, "x"), _dev(out, "out", (B, Cout, Tout)), B, Cin, Cout, T,
                             _dev(w, "w"), _opt(bias, "bias", (Cout,)), K, dilation, pad,
                             _opt(residual, "residual", (B, Cout, Tout)), _stream(stream)))
    return out


def conv1d_fft_pack(w, dilation: int = 1, out=None, stream=None):
    """avae_conv1d_fft_pack: w [Cout, Cin, K] -> packed frequency-domain weights."""
    torch = _torch()
    Cout, Cin, K = w.shape
    n = int(lib().avae_conv1d_fft_weight_floats(Cin, Cout))
    if out is None:
        out = torch.empty((n,), device=w.device, dtype=torch.float32)
    _check(lib().avae_conv1d_fft_pack(_dev(w, "w"), _dev(out, "out", (n,)), Cin, Cout, K,
                                      dilation, _stream(stream)))
    return out


def conv1d_fft_workspace_bytes(B: int, Cin: int, Cout: int, T: int, K: int,
                               dilation: int = 1) -> int:
    return int(lib().avae_conv1d_fft_workspace_bytes(B, Cin, Cout, T, K, dilation))


def conv1d_fft(x, wp, Cout: int, K: int, bias=None, dilation: int = 1, residual=None, out=None,
               workspace=None, stream=None):
    """avae_conv1d_fft: 'same'-padded Conv1d with weights packed by conv1d_fft_pack."""
    torch = _torch()
    B, Cin, T = x.shape
    if out is None:
        out = torch.empty((B, Cout, T), device=x.device, dtype=torch.float32)
    need = conv1d_fft_workspace_bytes(B, Cin, Cout, T, K, dilation)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), device=x.device, dtype=torch.uint8)
    if workspace.dtype != torch.uint8 or not workspace.is_cuda:
        raise ValueError("workspace must be a uint8 device tensor")
    _check(lib().avae_conv1d_fft(_dev(x, "x"), _dev(out, "out", (B, Cout, T)), B, Cin, Cout, T,
                                 _dev(wp, "wp"), _opt(bias, "bias", (Cout,)), K, dilation,
                                 _opt(residual, "residual", (B, Cout, T)),
                                 workspace.data_ptr(), workspace.numel(),
                                 _stream(stream)))
    return out


def act_conv1d_fft(x, log_alpha, log_beta, wp, Cout: int, K: int, bias=None, dilation: int = 1,
                   residual=None, out=None, workspace=None, stream=None):
    """avae_act_conv1d_fft: conv1d_fft of act1d(x) (designed taps), one pass."""
    torch = _torch()
    B, Cin, T = x.shape
    if out is None:
        out = torch.empty((B, Cout, T), device=x.device, dtype=torch.float32)
    need = conv1d_fft_workspace_bytes(B, Cin, Cout, T, K, dilation)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), device=x.device, dtype=torch.uint8)
    if workspace.dtype != torch.uint8 or not workspace.is_cuda:
        raise ValueError("workspace must be a uint8 device tensor")
    _check(lib().avae_act_conv1d_fft(
        _dev(x, "x"), _dev(out, "out", (B, Cout, T)), B, Cin, Cout, T,
        _dev(log_alpha, "log_alpha", (Cin,)), _dev(log_beta, "log_beta", (Cin,)), _dev(wp, "wp"),
        _opt(bias, "bias", (Cout,)), K, dilation, _opt(residual, "residual", (B, Cout, T)),
        workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return out


def convtr1d(x, w, bias=None, stride: int = 1, pad: int = -1, out=None, stream=None):
    """avae_convtr1d; pad < 0 selects (K - stride)/2."""
    torch = _torch()
    B, Cin, Tin = x.shape
    Cin_w, Cout, K = w.shape
    if Cin_w != Cin:
        raise ValueError(f"weight has {Cin_w} input channels, x has {Cin}")
    p = (K - stride) // 2 if pad < 0 else pad
    Tout = (Tin - 1) * stride + K - 2 * p
    if out is None:
        out = torch.empty((B, Cout, max(Tout, 0)), device=x.device, dtype=torch.float32)
    _check(lib().avae_convtr1d(_dev(x, "x"), _dev(out, "out", (B, Cout, Tout)), B, Cin, Cout, Tin,
                               _dev(w, "w"), _opt(bias, "bias", (Cout,)), K, stride, pad,
                               _stream(stream)))
    return out


def amp_block_workspace_bytes(B: int, C: int, T: int) -> int:
    return int(lib().avae_amp_block_workspace_bytes(B, C, T))


def amp_block_fft_workspace_bytes(B: int, C: int, T: int, K: int, dil: Sequence[int]) -> int:
    n = len(dil)
    dil_a = (c_int * n)(*[int(d) for d in dil])
    return int(lib().avae_amp_block_fft_workspace_bytes(B, C, T, K, n, ctypes.addressof(dil_a)))


def amp_block(x, K: int, dil: Sequence[int], w1: List, b1: List, w2: List, b2: List,
              log_alpha: List, log_beta: List, out_scale: float = 1.0, accumulate: bool = False,
              out=None, workspace=None, stream=None, fft: bool = True):
    """avae_amp_block: out = [out +] out_scale * AMP(x).  Without a workspace,
    one is allocated: sized for the frequency-domain convolutions if fft,
    else for the direct ones."""
    torch = _torch()
    B, C, T = x.shape
    n = len(dil)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out tensor")
        out = torch.empty_like(x)
    if workspace is None:
        nb = (amp_block_fft_workspace_bytes(B, C, T, K, dil) if fft
              else amp_block_workspace_bytes(B, C, T))
        workspace = torch.empty(nb, dtype=torch.uint8, device=x.device)
    dil_a = (c_int * n)(*[int(d) for d in dil])
    arr = lambda ts, nm, shape: (P * len(ts))(*[_opt(t, nm, shape) for t in ts])
    w1a = arr(w1, "w1", (C, C, K))
    b1a = arr(b1, "b1", (C,))
    w2a = arr(w2, "w2", (C, C, K))
    b2a = arr(b2, "b2", (C,))
    laa = arr(log_alpha, "log_alpha", (C,))
    lba = arr(log_beta, "log_beta", (C,))
    if len(w1) != n or len(w2) != n or len(log_alpha) != 2 * n or len(log_beta) != 2 * n:
        raise ValueError("amp_block: per-dilation lists have the wrong length")
    if workspace.dtype != torch.uint8 or not workspace.is_cuda:
        raise ValueError("workspace must be a uint8 device tensor")
    _check(lib().avae_amp_block(
        _dev(x, "x"), _dev(out, "out", (B, C, T)), B, C, T, K, n, ctypes.addressof(dil_a),
        ctypes.addressof(w1a), ctypes.addressof(b1a), ctypes.addressof(w2a),
        ctypes.addressof(b2a), ctypes.addressof(laa), ctypes.addressof(lba), float(out_scale),
        1 if accumulate else 0, workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return out


def amp_block_static_max_bytes() -> int:
    return int(lib().avae_amp_block_static_max_bytes())


def amp_block_static(x, K: int, dil: Sequence[int], w1: List, b1: List, w2: List, b2: List,
                     log_alpha: List, log_beta: List, out_scale: float = 1.0,
                     accumulate: bool = False, out=None, stream=None):
    """avae_amp_block_static: avae_amp_block with the library's static device
    scratch instead of a workspace (nothing is allocated by the library;
    `out` is allocated here only when the caller passes none)."""
    torch = _torch()
    B, C, T = x.shape
    n = len(dil)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out tensor")
        out = torch.empty_like(x)
    if len(w1) != n or len(w2) != n or len(log_alpha) != 2 * n or len(log_beta) != 2 * n:
        raise ValueError("amp_block_static: per-dilation lists have the wrong length")
    dil_a = (c_int * n)(*[int(d) for d in dil])
    arr = lambda ts, nm, shape: (P * len(ts))(*[_opt(t, nm, shape) for t in ts])
    w1a = arr(w1, "w1", (C, C, K))
    b1a = arr(b1, "b1", (C,))
    w2a = arr(w2, "w2", (C, C, K))
    b2a = arr(b2, "b2", (C,))
    laa = arr(log_alpha, "log_alpha", (C,))
    lba = arr(log_beta, "log_beta", (C,))
    _check(lib().avae_amp_block_static(
        _dev(x, "x"), _dev(out, "out", (B, C, T)), B, C, T, K, n, ctypes.addressof(dil_a),
        ctypes.addressof(w1a), ctypes.addressof(b1a), ctypes.addressof(w2a),
        ctypes.addressof(b2a), ctypes.addressof(laa), ctypes.addressof(lba), float(out_scale),
        1 if accumulate else 0, _stream(stream)))
    return out


def _decoder_structs(spec, tensors: Dict[str, "object"]):
    """avae_config and avae_weights of a BigVGAN decoder spec, weights named
    as on the H3 page."""
    cfg = avae_config()
    cfg.c_in = spec.c_in
    cfg.dec_in_ch = int(spec.dec_in)
    cfg.has_latent_affine = 1 if spec.latent_affine else 0
    cfg.k_pre, cfg.k_post = spec.k_pre, spec.k_post
    ns = len(spec.rates)
    if ns > AVAE_MAX_STAGES:
        raise ValueError("too many stages")
    cfg.n_stages = ns
    for i, c in enumerate(spec.widths()):
        cfg.ch[i] = c
    for i, (r, k) in enumerate(zip(spec.rates, spec.up_k)):
        cfg.rates[i], cfg.up_k[i] = r, k
    nk = len(spec.rb_k)
    cfg.n_kernels = nk
    nd = len(spec.rb_d[0])
    cfg.n_dil = nd
    for j in range(nk):
        cfg.rb_k[j] = spec.rb_k[j]
        if len(spec.rb_d[j]) != nd:
            raise ValueError("every AMP block needs the same number of dilations")
        for q in range(nd):
            cfg.rb_d[j][q] = spec.rb_d[j][q]
    cfg.final_act = FINAL[spec.final]
    t = tensors
    g = lambda name: _dev(t[name], name) if name in t else None
    w = avae_weights()
    w.latent_mean, w.latent_std = g("latents_mean"), g("latents_std")
    w.dec_in_w, w.dec_in_b = g("dec_in.weight"), g("dec_in.bias")
    w.conv_pre_w, w.conv_pre_b = g("conv_pre.weight"), g("conv_pre.bias")
    for i in range(ns):
        w.up_w[i], w.up_b[i] = g(f"ups.{i}.weight"), g(f"ups.{i}.bias")
        for j in range(nk):
            p = f"resblocks.{i * nk + j}"
            for q in range(nd):
                w.w1[i][j][q] = g(f"{p}.convs1.{q}.weight")
                w.b1[i][j][q] = g(f"{p}.convs1.{q}.bias")
                w.w2[i][j][q] = g(f"{p}.convs2.{q}.weight")
                w.b2[i][j][q] = g(f"{p}.convs2.{q}.bias")
            for q in range(2 * nd):
                w.act_la[i][j][q] = g(f"{p}.activations.{q}.act.alpha")
                w.act_lb[i][j][q] = g(f"{p}.activations.{q}.act.beta")
    w.post_la, w.post_lb = g("activation_post.act.alpha"), g("activation_post.act.beta")
    w.conv_post_w, w.conv_post_b = g("conv_post.weight"), g("conv_post.bias")
    return cfg, w


class Decoder:
    """avae_decoder_create / avae_bigvgan_decode over device weight tensors
    named as on the H3 page (``conv_pre.weight``, ``ups.{i}.weight``,
    ``resblocks.{i*nk+j}.convs1.{q}.weight``,
    ``resblocks.{..}.activations.{q}.act.alpha`` ...)."""

    def __init__(self, spec, tensors: Dict[str, "object"]):
        cfg, w = _decoder_structs(spec, tensors)
        self.spec = spec
        self.cfg = cfg
        h = P()
        _check(lib().avae_decoder_create(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h)))
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:
            _lib.avae_decoder_destroy(h)
            self._h = None

    def output_length(self, frames: int) -> int:
        n = c_int()
        _check(lib().avae_decoder_output_length(self._h, frames, ctypes.byref(n)))
        return n.value

    def workspace_bytes(self, B: int, frames: int) -> int:
        return int(lib().avae_decoder_workspace_bytes(self._h, B, frames))

    def set_concurrent(self, on: bool) -> None:
        """Run a stage's AMP blocks overlapped on side streams (default) or
        one after the other on the caller's stream."""
        _check(lib().avae_decoder_set_concurrent(self._h, 1 if on else 0))

    def stage_shapes(self, B: int, frames: int):
        """Shapes of the traced intermediates (conv_pre, each stage, pre-final)."""
        w = self.spec.widths()
        shapes = [(B, w[0], frames)]
        T = frames
        for i, (r, k) in enumerate(zip(self.spec.rates, self.spec.up_k)):
            T = (T - 1) * r + k - 2 * ((k - r) // 2)
            shapes.append((B, w[i + 1], T))
        shapes.append((B, self.output_length(frames)))
        return shapes

    def decode(self, latent, out=None, workspace=None, stream=None, trace: bool = False):
        """latent [B, c_in, F] -> wave [B, L]; with trace=True also returns
        the list of intermediates."""
        torch = _torch()
        B, C, F = latent.shape
        if C != self.spec.c_in:
            raise ValueError(f"latent has {C} channels, decoder expects {self.spec.c_in}")
        L = self.output_length(F)
        if out is None:
            out = torch.empty((B, L), device=latent.device, dtype=torch.float32)
        if workspace is None:
            workspace = torch.empty(self.workspace_bytes(B, F), dtype=torch.uint8,
                                    device=latent.device)
        if workspace.dtype != torch.uint8 or not workspace.is_cuda:
            raise ValueError("workspace must be a uint8 device tensor")
        if not trace:
            _check(lib().avae_bigvgan_decode(self._h, _dev(latent, "latent"), B, F,
                                             _dev(out, "out", (B, L)), workspace.data_ptr(),
                                             workspace.numel(), _stream(stream)))
            return out
        stages = [torch.empty(s, device=latent.device, dtype=torch.float32)
                  for s in self.stage_shapes(B, F)]
        arr = (P * len(stages))(*[s.data_ptr() for s in stages])
        _check(lib().avae_bigvgan_decode_traced(self._h, _dev(latent, "latent"), B, F,
                                                _dev(out, "out", (B, L)), workspace.data_ptr(),
                                                workspace.numel(), ctypes.addressof(arr),
                                                _stream(stream)))
        return out, stages

    def reach_frames(self) -> int:
        n = c_int()
        _check(lib().avae_decoder_reach_frames(self._h, ctypes.byref(n)))
        return n.value

    def streaming_workspace_bytes(self, B: int, tile_frames: int, halo_frames: int = -1) -> int:
        return int(lib().avae_decoder_streaming_workspace_bytes(self._h, B, tile_frames,
                                                                  halo_frames))

    def decode_streaming(self, latent, tile_frames: int, halo_frames: int = -1, out=None,
                         workspace=None, stream=None):
        """avae_bigvgan_decode_streaming: latent [B, c_in, F] -> wave [B, F*hop] in
        tiles of tile_frames frames (halo < 0: the decoder's receptive-field reach)."""
        torch = _torch()
        B, C, F = latent.shape
        if C != self.spec.c_in:
            raise ValueError(f"latent has {C} channels, decoder expects {self.spec.c_in}")
        L = F * self.spec.hop
        if out is None:
            out = torch.empty((B, L), device=latent.device, dtype=torch.float32)
        if workspace is None:
            workspace = torch.empty(self.streaming_workspace_bytes(B, min(tile_frames, F),
                                                                   halo_frames),
                                    dtype=torch.uint8, device=latent.device)
        _check(lib().avae_bigvgan_decode_streaming(
            self._h, _dev(latent, "latent"), B, F, _dev(out, "out", (B, L)), int(tile_frames),
            int(halo_frames), workspace.data_ptr(), workspace.numel(), _stream(stream)))
        return out



def probe_mfma(chains: int, blocks: int, iters: int, sink, stream=None) -> None:
    """avae_probe_mfma: a pure FP32-MFMA loop (measurement aid); the caller
    times it.  flops = blocks * 4 * iters * chains * 2048."""
    _check(lib().avae_probe_mfma(chains, blocks, iters, _dev(sink, "sink", (blocks * 256,)),
                                 _stream(stream)))

def probe_copy(x, out, stream=None) -> None:
    """avae_probe_copy: out = x by a streaming float4 copy (measurement
    aid); the caller times it.  bytes moved = 8 * x.numel()."""
    n = x.numel()
    _check(lib().avae_probe_copy(_dev(x, "x"), _dev(out, "out", tuple(x.shape)), n,
                                 _stream(stream)))


def snake(x, alpha, out=None, stream=None):
    """avae_snake: plain Snake with alpha as stored; out may be x."""
    torch = _torch()
    B, C, T = x.shape
    if out is None:
        out = torch.empty_like(x)
    _check(lib().avae_snake(_dev(x, "x"), _dev(out, "out", (B, C, T)), B, C, T,
                            _dev(alpha, "alpha", (C,)), _stream(stream)))
    return out


class DavDecoder:
    """avae_dav_create / avae_dav_decode over device weight tensors named as on
    the H3 page (``mvae.dec_in_proj.weight``, ``mvae.decoder.model.{i}...``)."""

    def __init__(self, spec, tensors: Dict[str, "object"]):
        cfg = avae_dav_config()
        cfg.c_side, cfg.dec_in_ch = spec.c_side, spec.dec_in
        cfg.k_pre, cfg.k_post = spec.k_pre, spec.k_post
        ns = len(spec.strides)
        cfg.n_stages = ns
        for i, c in enumerate(spec.widths()):
            cfg.ch[i] = c
        for i, (st, k) in enumerate(zip(spec.strides, spec.up_k)):
            cfg.strides[i], cfg.up_k[i] = st, k
        cfg.unit_k = spec.unit_k
        cfg.n_units = len(spec.unit_dil)
        for u, d in enumerate(spec.unit_dil):
            cfg.unit_dil[u] = d
        self.spec, self.cfg = spec, cfg
        t = tensors
        g = lambda name: _dev(t[name], name) if name in t else None
        w = avae_dav_weights()
        w.dec_in_w, w.dec_in_b = g("mvae.dec_in_proj.weight"), g("mvae.dec_in_proj.bias")
        w.conv_pre_w, w.conv_pre_b = g("mvae.decoder.model.0.weight"), g("mvae.decoder.model.0.bias")
        for i in range(ns):
            p = f"mvae.decoder.model.{i + 1}"
            w.stage_alpha[i] = g(f"{p}.block.0.alpha")
            w.up_w[i], w.up_b[i] = g(f"{p}.block.1.weight"), g(f"{p}.block.1.bias")
            for u in range(len(spec.unit_dil)):
                q = f"{p}.block.{u + 2}"
                w.a1[i][u] = g(f"{q}.block.0.alpha")
                w.w1[i][u], w.b1[i][u] = g(f"{q}.block.1.weight"), g(f"{q}.block.1.bias")
                w.a2[i][u] = g(f"{q}.block.2.alpha")
                w.w2[i][u], w.b2[i][u] = g(f"{q}.block.3.weight"), g(f"{q}.block.3.bias")
        w.post_alpha = g(f"mvae.decoder.model.{ns + 1}.alpha")
        w.conv_post_w = g(f"mvae.decoder.model.{ns + 2}.weight")
        w.conv_post_b = g(f"mvae.decoder.model.{ns + 2}.bias")
        h = P()
        _check(lib().avae_dav_create(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h)))
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:
            _lib.avae_dav_destroy(h)
            self._h = None

    def output_length(self, frames: int) -> int:
        """Samples per side."""
        n = c_int()
        _check(lib().avae_dav_output_length(self._h, frames, ctypes.byref(n)))
        return n.value

    def workspace_bytes(self, B: int, frames: int) -> int:
        return int(lib().avae_dav_workspace_bytes(self._h, B, frames))

    def stage_shapes(self, B: int, frames: int):
        """Traced intermediates of the [2B, ...] side batch."""
        w = self.spec.widths()
        shapes = [(2 * B, w[0], frames)]
        T = frames
        for i, (st, k) in enumerate(zip(self.spec.strides, self.spec.up_k)):
            T = (T - 1) * st + k - 2 * ((k - st) // 2)
            shapes.append((2 * B, w[i + 1], T))
        shapes.append((2 * B, self.output_length(frames)))
        return shapes

    def decode(self, latent, out=None, workspace=None, stream=None, trace: bool = False):
        """latent [B, 2 c_side, F] -> interleaved stereo [B, 2 L]."""
        torch = _torch()
        B, C, F = latent.shape
        if C != 2 * self.spec.c_side:
            raise ValueError(f"latent has {C} channels, the DAV decoder expects "
                             f"{2 * self.spec.c_side} (two sides)")
        L = self.output_length(F)
        if out is None:
            out = torch.empty((B, 2 * L), device=latent.device, dtype=torch.float32)
        if workspace is None:
            workspace = torch.empty(self.workspace_bytes(B, F), dtype=torch.uint8,
                                    device=latent.device)
        if not trace:
            _check(lib().avae_dav_decode(self._h, _dev(latent, "latent"), B, F,
                                         _dev(out, "out", (B, 2 * L)), workspace.data_ptr(),
                                         workspace.numel(), _stream(stream)))
            return out
        stages = [torch.empty(s, device=latent.device, dtype=torch.float32)
                  for s in self.stage_shapes(B, F)]
        arr = (P * len(stages))(*[s.data_ptr() for s in stages])
        _check(lib().avae_dav_decode_traced(self._h, _dev(latent, "latent"), B, F,
                                            _dev(out, "out", (B, 2 * L)), workspace.data_ptr(),
                                            workspace.numel(), ctypes.addressof(arr),
                                            _stream(stream)))
        return out, stages


def mel_stft(x, forward_basis, mel_basis, hop: int, out=None, stream=None):
    """avae_mel_stft: x [B, T] -> causal log-mel [B, n_mels, T // hop]."""
    torch = _torch()
    B, T = x.shape
    nf2, L = forward_basis.shape
    n_mels, nf = mel_basis.shape
    if nf2 != 2 * nf:
        raise ValueError("forward_basis needs 2 n_freqs rows")
    frames = T // hop
    if out is None:
        out = torch.empty((B, n_mels, frames), device=x.device, dtype=torch.float32)
    _check(lib().avae_mel_stft(_dev(x, "x"), _dev(out, "out", (B, n_mels, frames)), B, T,
                               _dev(forward_basis, "forward_basis"), nf, L, hop,
                               _dev(mel_basis, "mel_basis"), n_mels, _stream(stream)))
    return out


def hann_sinc_upsample(x, ratio: int = 3, out=None, stream=None):
    """avae_hann_sinc_upsample: x [B, T] -> [B, ratio T]."""
    torch = _torch()
    B, T = x.shape
    if out is None:
        out = torch.empty((B, ratio * T), device=x.device, dtype=torch.float32)
    _check(lib().avae_hann_sinc_upsample(_dev(x, "x"), _dev(out, "out", (B, ratio * T)), B, T,
                                         ratio, _stream(stream)))
    return out


class BweDecoder:
    """avae_bwe_create / avae_bwe_decode: the bandwidth-extension tail, the
    generator's weights named as for Decoder, the bases as
    ``mel_stft.forward_basis`` [2 nf, L] and ``mel_stft.mel_basis`` [n_mels, nf]."""

    def __init__(self, spec, tensors: Dict[str, "object"], hop: int = 80, ratio: int = 3):
        gcfg, gw = _decoder_structs(spec, tensors)
        fb, mb = tensors["mel_stft.forward_basis"], tensors["mel_stft.mel_basis"]
        cfg = avae_bwe_config()
        cfg.gen = gcfg
        cfg.filter_len, cfg.hop, cfg.ratio = fb.shape[1], hop, ratio
        cfg.n_mels, cfg.n_freqs = mb.shape
        w = avae_bwe_weights()
        w.gen = gw
        w.forward_basis, w.mel_basis = _dev(fb, "forward_basis"), _dev(mb, "mel_basis")
        self.spec, self.cfg = spec, cfg
        h = P()
        _check(lib().avae_bwe_create(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(h)))
        self._h = h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:
            _lib.avae_bwe_destroy(h)
            self._h = None

    def workspace_bytes(self, B: int, T: int) -> int:
        return int(lib().avae_bwe_workspace_bytes(self._h, B, T))

    def decode(self, low, out=None, workspace=None, stream=None, trace: bool = False):
        """low [B, T] at the input rate -> [B, ratio T]; trace=True also
        returns the log-mel and the generator's residual."""
        torch = _torch()
        B, T = low.shape
        r, hop = self.cfg.ratio, self.cfg.hop
        if out is None:
            out = torch.empty((B, r * T), device=low.device, dtype=torch.float32)
        if workspace is None:
            workspace = torch.empty(self.workspace_bytes(B, T), dtype=torch.uint8,
                                    device=low.device)
        if not trace:
            _check(lib().avae_bwe_decode(self._h, _dev(low, "low"), B, T,
                                         _dev(out, "out", (B, r * T)), workspace.data_ptr(),
                                         workspace.numel(), _stream(stream)))
            return out
        frames = -(-T // hop)
        mel = torch.empty((B, self.cfg.n_mels, frames), device=low.device, dtype=torch.float32)
        res = torch.empty((B, frames * hop * r), device=low.device, dtype=torch.float32)
        _check(lib().avae_bwe_decode_traced(self._h, _dev(low, "low"), B, T,
                                            _dev(out, "out", (B, r * T)), workspace.data_ptr(),
                                            workspace.numel(), mel.data_ptr(), res.data_ptr(),
                                            _stream(stream)))
        return out, mel, res


# ------------------------------------------------------------------ 8-bit serving operators
#
# These calls take a few microseconds on the device, so what the binding does
# for each of them counts: names are looked up once, and a tensor is asked
# for its properties once.
#
# A call runs on the current stream, or on `stream` (a torch stream): then all
# of it does, what it allocates included, so that no memory of the current
# stream is written or given back while the other one still works.  Outputs
# belong to that stream, as with torch's own operators under it.

ACT = {"none": 0, "silu": 1}


class _Env:
    """torch, the library's functions and the types, looked up once."""

    def __init__(self):
        torch = _torch()
        L = lib()
        self.strided = torch.empty_strided  # the quickest of the allocators to call
        self.int8, self.int32, self.uint8 = torch.int8, torch.int32, torch.uint8
        self.float32 = torch.float32
        self.codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
        self.raw_stream = torch._C._cuda_getCurrentRawStream
        self.device = torch._C._cuda_getDevice
        self.norm, self.quant, self.dequant = (L.avae_rms_norm_q8, L.avae_quant_q8,
                                               L.avae_dequant_q8)
        self.linear, self.linear_ws = L.avae_linear_q8, L.avae_linear_q8_workspace_bytes
        self.write, self.read = L.avae_kv_write_q8, L.avae_kv_read_q8
        self.attn, self.attn_ws = L.avae_attn_q8, L.avae_attn_q8_workspace_bytes
        self.qk, self.write_rope, self.tree = (L.avae_qk_norm_rope, L.avae_kv_write_rope_q8,
                                               L.avae_tree_mask)
        self.rules, self.rules_ws = L.avae_attn_rules_q8, L.avae_attn_rules_q8_workspace_bytes

    def vec(self, n, dtype, dev):
        return self.strided((n,), (1,), dtype=dtype, device=dev)

    def mat(self, m, n, dtype, dev):
        return self.strided((m, n), (n, 1), dtype=dtype, device=dev)

    def heads(self, t, h, d, dtype, dev):
        return self.strided((t, h, d), (h * d, d, 1), dtype=dtype, device=dev)

    def code(self, dtype) -> int:
        code = self.codes.get(dtype)
        if code is None:
            raise ValueError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
        return code

    def stream(self, t):
        """The raw stream to launch on: the current one of the tensor's device."""
        return self.raw_stream(t.get_device())


_env: Optional[_Env] = None


def _q8() -> _Env:
    global _env
    if _env is None:
        _env = _Env()
    return _env


def _bad(t, name: str, dtype, expected: str):
    """Says what is wrong with a tensor that a check refused."""
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name}: expected {expected} with the last axis contiguous, got "
                     f"{tuple(t.shape)} at strides {t.stride()}")


def _rows(t, name: str, dtype, rows: int, cols: int):
    """Pointer and row stride of a [rows, cols] device tensor whose last axis
    is contiguous."""
    if not t.is_cuda or t.dtype != dtype or t.shape != (rows, cols):
        _bad(t, name, dtype, f"[{rows}, {cols}]")
    ld, one = t.stride()
    if one != 1 and cols > 1:
        _bad(t, name, dtype, f"[{rows}, {cols}]")
    # the stride of a single row says nothing; torch may give any
    return t.data_ptr(), (ld if rows > 1 else cols)


def _vec(t, name: str, n: int, dtype):
    if not t.is_cuda or t.dtype != dtype or t.shape != (n,) or not t.is_contiguous():
        _bad(t, name, dtype, f"[{n}]")
    return t.data_ptr()


def _two_axes(t, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected two axes, got {tuple(t.shape)}")
    return t.shape


def rms_norm_q8(x, weight, eps: float = 1e-6, residual=None, stream=None):
    """avae_rms_norm_q8: x [M, C] (+ residual) -> (q [M, C] int8, scale [M],
    the sum in x's dtype or None)."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return rms_norm_q8(x, weight, eps, residual)
    E = _q8()
    M, C = _two_axes(x, "x")
    dtype, dev = x.dtype, x.device
    code = E.code(dtype)
    px, ldx = _rows(x, "x", dtype, M, C)
    q = E.mat(M, C, E.int8, dev)
    scale = E.vec(M, E.float32, dev)
    pr, ldr, total, pt = None, 0, None, None
    if residual is not None:
        pr, ldr = _rows(residual, "residual", dtype, M, C)
        total = E.mat(M, C, dtype, dev)
        pt = total.data_ptr()
    rc = E.norm(px, ldx, pr, ldr, _vec(weight, "weight", C, E.float32), M, C, code, eps, pt, C,
                q.data_ptr(), C, scale.data_ptr(), E.stream(x))
    if rc:
        _check(rc)
    return q, scale, total


def quant_q8(x, stream=None):
    """avae_quant_q8: x [M, C] -> (q [M, C] int8, scale [M])."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return quant_q8(x)
    E = _q8()
    M, C = _two_axes(x, "x")
    code = E.code(x.dtype)
    px, ldx = _rows(x, "x", x.dtype, M, C)
    q = E.mat(M, C, E.int8, x.device)
    scale = E.vec(M, E.float32, x.device)
    rc = E.quant(px, ldx, M, C, code, q.data_ptr(), C, scale.data_ptr(), E.stream(x))
    if rc:
        _check(rc)
    return q, scale


def dequant_q8(q, scale, dtype=None, stream=None):
    """avae_dequant_q8: q [M, C] int8 with a scale a row -> [M, C] of dtype
    (float32 if none is given)."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return dequant_q8(q, scale, dtype)
    E = _q8()
    dtype = E.float32 if dtype is None else dtype
    M, C = _two_axes(q, "q")
    code = E.code(dtype)
    pq, ldq = _rows(q, "q", E.int8, M, C)
    y = E.mat(M, C, dtype, q.device)
    rc = E.dequant(pq, ldq, _vec(scale, "scale", M, E.float32), M, C, code, y.data_ptr(), C,
                   E.stream(q))
    if rc:
        _check(rc)
    return y


def linear_q8(a, a_scale, w, w_scale, bias=None, act: str = "none", dtype=None, stream=None):
    """avae_linear_q8: a [M, K] int8, w [N, K] int8 with a scale a row each
    -> [M, N] of dtype (float32 if none is given)."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return linear_q8(a, a_scale, w, w_scale, bias, act, dtype)
    E = _q8()
    dtype = E.float32 if dtype is None else dtype
    M, K = _two_axes(a, "a")
    N = _two_axes(w, "w")[0]
    code, act_code = E.code(dtype), ACT.get(act)
    if act_code is None:
        raise ValueError(f"act must be one of {sorted(ACT)}, got {act!r}")
    pa, lda = _rows(a, "a", E.int8, M, K)
    pw, ldw = _rows(w, "w", E.int8, N, K)
    y = E.mat(M, N, dtype, a.device)
    need = E.linear_ws(M, N, K)
    ws = E.vec(need, E.uint8, a.device) if need else None
    rc = E.linear(pa, lda, _vec(a_scale, "a_scale", M, E.float32), pw, ldw,
                  _vec(w_scale, "w_scale", N, E.float32),
                  None if bias is None else _vec(bias, "bias", N, E.float32), M, N, K, act_code,
                  code, y.data_ptr(), N, None if ws is None else ws.data_ptr(), need,
                  E.stream(a))
    if rc:
        _check(rc)
    return y


class KvCacheQ8:
    """The four tensors of a paged 8-bit cache (avae_kv_q8): k, v [n_pages,
    heads, page, dim] int8 and k_scale, v_scale [n_pages, heads] float32."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "heads", "page", "dim", "c", "ref")

    def __init__(self, k, v, k_scale, v_scale):
        E = _q8()
        if k.dim() != 4:
            raise ValueError(f"k: expected [n_pages, heads, page, dim], got {tuple(k.shape)}")
        shape, i8, f32 = k.shape, E.int8, E.float32
        scales = shape[:2]
        if not (k.is_cuda and k.dtype is i8 and k.is_contiguous()):
            _bad(k, "k", i8, f"{tuple(shape)}")
        if not (v.is_cuda and v.dtype is i8 and v.shape == shape and v.is_contiguous()):
            _bad(v, "v", i8, f"{tuple(shape)}")
        if not (k_scale.is_cuda and k_scale.dtype is f32 and k_scale.shape == scales
                and k_scale.is_contiguous()):
            _bad(k_scale, "k_scale", f32, f"{tuple(scales)}")
        if not (v_scale.is_cuda and v_scale.dtype is f32 and v_scale.shape == scales
                and v_scale.is_contiguous()):
            _bad(v_scale, "v_scale", f32, f"{tuple(scales)}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        _, self.heads, self.page, self.dim = shape
        self.c = avae_kv_q8(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                            *shape)
        self.ref = ctypes.addressof(self.c)

    @classmethod
    def empty(cls, n_pages: int, heads: int, page: int, dim: int, device="cuda"):
        """A cache with no token in it (what it holds does not matter: a page
        is written from its first token on)."""
        torch = _torch()
        shape = (n_pages, heads, page, dim)
        return cls(*(torch.zeros(shape, dtype=torch.int8, device=device) for _ in range(2)),
                   *(torch.zeros(shape[:2], dtype=torch.float32, device=device) for _ in range(2)))


def _ragged(E, table, cu, lens, total: int, max_rows: Optional[int]):
    seqs, cols = _two_axes(table, "table")
    pt, ld = _rows(table, "table", E.int32, seqs, cols)
    return avae_ragged(_vec(cu, "cu", seqs + 1, E.int32), _vec(lens, "lens", seqs, E.int32), pt, ld,
                       cols, seqs, total,
                       total if max_rows is None or max_rows > total else max_rows)


def _heads(t, name: str, heads: Optional[int], dim: int):
    """Pointer, token and head stride of a [tokens, heads, dim] tensor."""
    if (not t.is_cuda or t.dim() != 3 or t.shape[2] != dim
            or (heads is not None and t.shape[1] != heads)):
        _bad(t, name, t.dtype, f"[tokens, {heads or 'heads'}, {dim}]")
    tok, head, one = t.stride()
    if one != 1:
        _bad(t, name, t.dtype, f"[tokens, {heads or 'heads'}, {dim}]")
    return t.data_ptr(), tok, head


def kv_write_q8(cache: KvCacheQ8, k, v, table, cu, lens, max_new: Optional[int] = None,
                stream=None):
    """avae_kv_write_q8: k, v [tokens, heads, dim] into the cache's pages.
    max_new: at least the most rows of one sequence (all of them if not given;
    the launch goes by it)."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return kv_write_q8(cache, k, v, table, cu, lens, max_new)
    E = _q8()
    total = k.shape[0]
    if v.dtype != k.dtype or v.shape[0] != total:
        raise ValueError("k and v must have one dtype and as many tokens")
    rows = _ragged(E, table, cu, lens, total, max_new)
    rc = E.write(*_heads(k, "k", cache.heads, cache.dim), *_heads(v, "v", cache.heads, cache.dim),
                 E.code(k.dtype), cache.ref, ctypes.addressof(rows), E.stream(k))
    if rc:
        _check(rc)


def kv_read_q8(cache: KvCacheQ8, table, cu, lens, total: int, max_rows: Optional[int] = None,
               dtype=None, stream=None):
    """avae_kv_read_q8: the sequences' last tokens, `total` of them, as cu
    says -> k, v [total, heads, dim] of dtype (float32 if none is given)."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return kv_read_q8(cache, table, cu, lens, total, max_rows, dtype)
    E = _q8()
    dtype = E.float32 if dtype is None else dtype
    code = E.code(dtype)
    dev = cache.k.device
    k = E.heads(total, cache.heads, cache.dim, dtype, dev)
    v = E.heads(total, cache.heads, cache.dim, dtype, dev)
    rows = _ragged(E, table, cu, lens, total, max_rows)
    rc = E.read(cache.ref, ctypes.addressof(rows), code, k.data_ptr(), v.data_ptr(),
                E.stream(cache.k))
    if rc:
        _check(rc)
    return k, v


def attn_q8(q, cache: KvCacheQ8, table, cu, lens, max_q: Optional[int] = None,
            max_len: Optional[int] = None, scale: Optional[float] = None, causal: bool = True,
            window: int = 0, first=None, return_lse: bool = False, stream=None):
    """avae_attn_q8: q [tokens, q_heads, dim] over the cache -> the same shape
    (and lse [tokens, q_heads] float32 if asked for).  max_q: at least the most
    rows of one sequence (all of them if not given, which is slow for many
    short ones: the kernel is chosen by it); max_len: at least the longest
    sequence (the table's tokens if not given); scale: 1 / sqrt(dim) if not
    given."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return attn_q8(q, cache, table, cu, lens, max_q, max_len, scale, causal, window, first,
                           return_lse)
    E = _q8()
    dim, dtype, dev = cache.dim, q.dtype, q.device
    code = E.code(dtype)
    pq, tok, head = _heads(q, "q", None, dim)
    total, heads, _ = q.shape
    rows = _ragged(E, table, cu, lens, total, max_q)
    pr = ctypes.addressof(rows)
    if max_len is None:
        max_len = rows.table_cols * cache.page
    out = E.heads(total, heads, dim, dtype, dev)
    lse = E.mat(total, heads, E.float32, dev) if return_lse else None
    need = E.attn_ws(cache.ref, pr, heads, code, max_len, window)
    ws = E.vec(need, E.uint8, dev) if need else None
    rc = E.attn(pq, tok, head, heads, code, cache.ref, pr,
                None if first is None else _vec(first, "first", rows.seqs, E.int32), max_len,
                dim ** -0.5 if scale is None else scale, 1 if causal else 0, window,
                out.data_ptr(), None if lse is None else lse.data_ptr(),
                None if ws is None else ws.data_ptr(), need, E.stream(q))
    if rc:
        _check(rc)
    return (out, lse) if return_lse else out


ROPE_SCALING = {"plain": 0, "linear": 1, "base": 2, "bands": 3, "ramp": 4}


def rope_freq(rot: int, theta: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
              context: float = 4096.0, low: float = 1.0, high: float = 32.0):
    """avae_rope_freq: (frequencies [rot / 2] float32 on the host, amp)."""
    kind = ROPE_SCALING.get(scaling)
    if kind is None:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALING)}, got {scaling!r}")
    freq, amp = np.empty(max(rot // 2, 1), np.float32), c_float()
    _check(lib().avae_rope_freq(rot, theta, kind, factor, context, low, high, freq.ctypes.data,
                                ctypes.addressof(amp)))
    return freq, amp.value


class Rope:
    """What turns queries and keys (avae_rope): freq [rot / 2] float32 on the
    device, radians a position.  Rope.of(rot, ..) takes rope_freq's."""

    __slots__ = ("freq", "rot", "c", "ref")

    def __init__(self, freq, interleaved: bool = False, amp: float = 1.0):
        shape = freq.shape
        if len(shape) != 1 or shape[0] < 1:
            raise ValueError(f"freq: expected [rot / 2], got {tuple(shape)}")
        if not (freq.is_cuda and freq.dtype is _q8().float32 and freq.is_contiguous()):
            _bad(freq, "freq", _q8().float32, f"[{shape[0]}]")
        self.freq, self.rot = freq, 2 * shape[0]
        self.c = avae_rope(freq.data_ptr(), self.rot, 1 if interleaved else 0, amp)
        self.ref = ctypes.addressof(self.c)

    @classmethod
    def of(cls, rot: int, interleaved: bool = False, device="cuda", **kw):
        freq, amp = rope_freq(rot, **kw)
        return cls(_torch().from_numpy(freq).to(device), interleaved, amp)


# The checks of the calls below: as those above, and that every tensor is on
# the first one's device.

def _bad_at(t, name: str, dtype, dev: int, expected: str):
    if t.is_cuda and t.get_device() != dev:
        raise ValueError(f"{name}: on device {t.get_device()}, the first tensor on {dev}")
    _bad(t, name, dtype, expected)


def _vec_at(t, name: str, n: int, dtype, dev: int):
    if (t.get_device() != dev or t.dtype is not dtype or t.shape != (n,)
            or not t.is_contiguous() or dev < 0):
        _bad_at(t, name, dtype, dev, f"[{n}]")
    return t.data_ptr()


def _heads_at(t, name: str, dtype, total: int, heads: Optional[int], dim: int, dev: int):
    """Pointer, token and head stride of a [total, heads, dim] tensor."""
    shape = t.shape
    if (len(shape) != 3 or shape[0] != total or shape[2] != dim or t.dtype is not dtype
            or t.get_device() != dev or dev < 0 or (heads is not None and shape[1] != heads)):
        _bad_at(t, name, dtype, dev, f"[{total}, {heads or 'heads'}, {dim}]")
    tok, head, one = t.stride()
    if one != 1:
        _bad_at(t, name, dtype, dev, f"[{total}, {heads or 'heads'}, {dim}]")
    return t.data_ptr(), tok, head


def _rows_at(E, table, cu, lens, total: int, max_rows: Optional[int], dev: int):
    """Packed rows of sequences, with their pages or (table None) without."""
    i32 = E.int32
    (seqs,) = lens.shape
    pt, ld, cols = None, 0, 0
    if table is not None:
        shape = table.shape
        if len(shape) != 2 or shape[0] != seqs or table.dtype is not i32 or table.get_device() != dev:
            _bad_at(table, "table", i32, dev, f"[{seqs}, pages]")
        cols = shape[1]
        ld, one = table.stride()
        if one != 1 and cols > 1:
            _bad_at(table, "table", i32, dev, f"[{seqs}, pages]")
        # the stride of a single row says nothing; torch may give any
        pt, ld = table.data_ptr(), (ld if seqs > 1 else cols)
    return avae_ragged(_vec_at(cu, "cu", seqs + 1, i32, dev), _vec_at(lens, "lens", seqs, i32, dev), pt,
                       ld, cols, seqs, total,
                       total if max_rows is None or max_rows > total else max_rows)


_MOST = 2 ** 31 - 1


def _same_device(cache, dev: int):
    if cache.k.get_device() != dev:
        raise ValueError(f"the cache is on device {cache.k.get_device()}, the first tensor on {dev}")


def _freq_at(rope: Optional[Rope], dev: int):
    if rope is None:
        return None
    if rope.freq.get_device() != dev:
        raise ValueError(f"the frequencies are on device {rope.freq.get_device()}, the first tensor "
                         f"on {dev}")
    return rope.ref


def qk_norm_rope(q, k, rope: Optional[Rope], q_weight=None, k_weight=None, eps: float = 1e-6,
                 positions=None, cu=None, lens=None, max_rows: Optional[int] = None,
                 inplace: bool = False, stream=None):
    """avae_qk_norm_rope: q [tokens, q_heads, dim] and k [tokens, k_heads, dim]
    (or None) -> both normed (with weights [dim]) and turned; k's place holds
    None if k is None.  A token's position is positions [tokens] int32, else
    its place as cu and lens say; one of the two is needed."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return qk_norm_rope(q, k, rope, q_weight, k_weight, eps, positions, cu, lens, max_rows,
                                inplace)
    E = _q8()
    dev = q.get_device()
    if dev >= 0 and dev != E.device():
        with _torch().cuda.device(dev):
            return qk_norm_rope(q, k, rope, q_weight, k_weight, eps, positions, cu, lens, max_rows,
                                inplace)
    if q.dim() != 3:
        raise ValueError(f"q: expected [tokens, heads, dim], got {tuple(q.shape)}")
    total, heads, dim = q.shape
    dtype, f32 = q.dtype, E.float32
    code = E.code(dtype)
    pq, q_tok, q_head = _heads_at(q, "q", dtype, total, heads, dim, dev)
    device = q.device
    pk = pko = k_out = None
    k_heads = k_tok = k_head = ko_tok = ko_head = 0
    if k is not None:
        pk, k_tok, k_head = _heads_at(k, "k", dtype, total, None, dim, dev)
        k_heads = k.shape[1]
        if inplace:
            k_out, pko, ko_tok, ko_head = k, pk, k_tok, k_head
        else:
            k_out = E.heads(total, k_heads, dim, dtype, device)
            pko, ko_tok, ko_head = k_out.data_ptr(), k_heads * dim, dim
    if inplace:
        q_out, pqo, qo_tok, qo_head = q, pq, q_tok, q_head
    else:
        q_out = E.heads(total, heads, dim, dtype, device)
        pqo, qo_tok, qo_head = q_out.data_ptr(), heads * dim, dim
    if (cu is None) != (lens is None):
        raise ValueError("cu and lens are given together or not at all")
    rows = None if cu is None else _rows_at(E, None, cu, lens, total, max_rows, dev)
    rc = E.qk(pq, q_tok, q_head, heads,
              None if q_weight is None else _vec_at(q_weight, "q_weight", dim, f32, dev),
              pk, k_tok, k_head, k_heads,
              None if k_weight is None else _vec_at(k_weight, "k_weight", dim, f32, dev), dim, code,
              eps, _freq_at(rope, dev),
              None if positions is None else _vec_at(positions, "positions", total, E.int32, dev),
              None if rows is None else ctypes.addressof(rows), total, pqo, qo_tok, qo_head, pko,
              ko_tok, ko_head, E.raw_stream(dev))
    if rc:
        _check(rc)
    return q_out, k_out


def kv_write_rope_q8(cache: KvCacheQ8, k, v, table, cu, lens, rope: Optional[Rope], k_weight=None,
                     eps: float = 1e-6, positions=None, max_new: Optional[int] = None,
                     stream=None):
    """avae_kv_write_rope_q8: kv_write_q8 with the keys normed (with k_weight
    [dim]) and turned on the way, by positions [tokens] int32 or their places."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return kv_write_rope_q8(cache, k, v, table, cu, lens, rope, k_weight, eps, positions,
                                    max_new)
    E = _q8()
    dev = k.get_device()
    if dev >= 0 and dev != E.device():
        with _torch().cuda.device(dev):
            return kv_write_rope_q8(cache, k, v, table, cu, lens, rope, k_weight, eps, positions,
                                    max_new)
    total, dtype = k.shape[0], k.dtype
    heads, dim = cache.heads, cache.dim
    _same_device(cache, dev)
    rows = _rows_at(E, table, cu, lens, total, max_new, dev)
    rc = E.write_rope(
        *_heads_at(k, "k", dtype, total, heads, dim, dev),
        *_heads_at(v, "v", dtype, total, heads, dim, dev), E.code(dtype),
        None if k_weight is None else _vec_at(k_weight, "k_weight", dim, E.float32, dev), eps,
        _freq_at(rope, dev),
        None if positions is None else _vec_at(positions, "positions", total, E.int32, dev),
        cache.ref, ctypes.addressof(rows), E.raw_stream(dev))
    if rc:
        _check(rc)


def _attn_rules(q, cache, table, cu, lens, max_q, max_len, scale, causal, window, first, rules,
                return_lse):
    E = _q8()
    dev = q.get_device()
    if dev >= 0 and dev != E.device():
        with _torch().cuda.device(dev):
            return _attn_rules(q, cache, table, cu, lens, max_q, max_len, scale, causal, window, first,
                               rules, return_lse)
    dim, dtype = cache.dim, q.dtype
    code = E.code(dtype)
    total = q.shape[0]
    pq, tok, head = _heads_at(q, "q", dtype, total, None, dim, dev)
    heads, device = q.shape[1], q.device
    _same_device(cache, dev)
    rows = _rows_at(E, table, cu, lens, total, max_q, dev)
    pr, px = ctypes.addressof(rows), ctypes.addressof(rules)
    if max_len is None:
        max_len = rows.table_cols * cache.page
    if window > _MOST or max_len > _MOST:  # ctypes would take their low 32 bits
        window, max_len = min(window, _MOST), min(max_len, _MOST)
    if rules.max_prefix < 0:
        rules.max_prefix = max_len
    out = E.heads(total, heads, dim, dtype, device)
    lse = E.mat(total, heads, E.float32, device) if return_lse else None
    need = E.rules_ws(cache.ref, pr, heads, code, max_len, window, px)
    ws = E.vec(need, E.uint8, device) if need else None
    rc = E.rules(pq, tok, head, heads, code, cache.ref, pr,
                 None if first is None else _vec_at(first, "first", rows.seqs, E.int32, dev),
                 max_len, dim ** -0.5 if scale is None else scale, 1 if causal else 0, window, px,
                 out.data_ptr(), None if lse is None else lse.data_ptr(),
                 None if ws is None else ws.data_ptr(), need, E.raw_stream(dev))
    if rc:
        _check(rc)
    return (out, lse) if return_lse else out


def attn_rules_q8(q, cache: KvCacheQ8, table, cu, lens, max_q: Optional[int] = None,
                  max_len: Optional[int] = None, scale: Optional[float] = None,
                  causal: bool = True, window: int = 0, first=None, cap: float = 0.0, slopes=None,
                  prefix=None, max_prefix: Optional[int] = None, return_lse: bool = False,
                  stream=None):
    """avae_attn_rules_q8: attn_q8 with scores capped (cap > 0), biased by
    distance (slopes [q_heads] float32), and the first prefix [seqs] int32
    tokens in view of every row.  max_prefix: at least the longest prefix
    (max_len if not given; beside a window, the keys are cut for as many)."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return attn_rules_q8(q, cache, table, cu, lens, max_q, max_len, scale, causal, window,
                                 first, cap, slopes, prefix, max_prefix, return_lse)
    E = _q8()
    if max_prefix is not None and max_prefix < 0:
        raise ValueError(f"max_prefix is not negative, got {max_prefix}")
    dev = q.get_device()
    rules = avae_attn_rules(
        cap, None if slopes is None else _vec_at(slopes, "slopes", q.shape[1], E.float32, dev),
        None if prefix is None else _vec_at(prefix, "prefix", lens.shape[0], E.int32, dev),
        -1 if max_prefix is None else min(max_prefix, _MOST), None, 0, 0)
    return _attn_rules(q, cache, table, cu, lens, max_q, max_len, scale, causal, window, first,
                       rules, return_lse)


def tree_mask(parents, cu, lens, max_rows: Optional[int] = None, stream=None):
    """avae_tree_mask: parents [tokens] int32 -> (mask [tokens, words] int32
    with a bit for each draft that a draft sees, positions [tokens] int32).
    max_rows: at least the most drafts of one sequence (all of the call's if
    not given), 4096 at most; the mask has a word for every 32 of them."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return tree_mask(parents, cu, lens, max_rows)
    E = _q8()
    if parents.dim() != 1:
        raise ValueError(f"parents: expected [tokens], got {tuple(parents.shape)}")
    total, dev, device = parents.shape[0], parents.get_device(), parents.device
    if dev >= 0 and dev != E.device():
        with _torch().cuda.device(dev):
            return tree_mask(parents, cu, lens, max_rows)
    p = _vec_at(parents, "parents", total, E.int32, dev)
    rows = _rows_at(E, None, cu, lens, total, max_rows, dev)
    words = (rows.max_rows + 31) // 32
    mask = E.mat(total, words, E.int32, device)
    positions = E.vec(total, E.int32, device)
    rc = E.tree(p, ctypes.addressof(rows), words, mask.data_ptr(), words, positions.data_ptr(),
                E.raw_stream(dev))
    if rc:
        _check(rc)
    return mask, positions


def attn_tree_q8(q, cache: KvCacheQ8, table, cu, lens, tree, max_q: Optional[int] = None,
                 max_len: Optional[int] = None, scale: Optional[float] = None, first=None,
                 cap: float = 0.0, return_lse: bool = False, stream=None):
    """avae_attn_rules_q8 over a tree of drafts: each row sees what lies before
    its sequence's rows, and of those rows the ones that its mask in tree
    [tokens, words] int32 has bits for (tree_mask makes it)."""
    if stream is not None:
        with _torch().cuda.stream(stream):
            return attn_tree_q8(q, cache, table, cu, lens, tree, max_q, max_len, scale, first, cap,
                                return_lse)
    E = _q8()
    total, words = q.shape[0], _two_axes(tree, "tree")[1]
    p, ld = _rows(tree, "tree", E.int32, total, words)
    if tree.get_device() != q.get_device():
        _bad_at(tree, "tree", E.int32, q.get_device(), f"[{total}, {words}]")
    rules = avae_attn_rules(cap, None, None, 0, p, ld, words)
    return _attn_rules(q, cache, table, cu, lens, max_q, max_len, scale, True, 0, first, rules,
                       return_lse)
