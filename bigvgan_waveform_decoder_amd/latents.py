"""An autoregressive latent generator on the 8-bit serving operators: the kind
of network that writes a decoder's latent frames one after the other, with
random weights as an example of how the operators run together.

    gen = LatentGenerator(Config(c_latent=32), weights, streams=2, max_frames=400)
    latent = gen.generate(prompts, frames=400)      # [2, 32, 400]
    wave = avae.Decoder(W.H3, decoder_weights).decode(latent)

A layer is: RMS norm of the residual stream (8-bit rows out), the packed
query, key and value product, the write of the new keys and values into the
8-bit paged cache, attention over it, the output product; then the norm again
and the two products of the feed-forward block.  Every product takes 8-bit
rows and weights; the residual stream and what lies between two operators is
bfloat16.  A step of one frame a stream and a prompt of many run the same
calls.

``python -m bigvgan_waveform_decoder_amd.latents`` generates latents, decodes
them and prints the times.
"""
from __future__ import annotations

import dataclasses
import math
from typing import Dict, List, Sequence

import torch

from . import avae


@dataclasses.dataclass(frozen=True)
class Config:
    c_latent: int = 32
    width: int = 1536
    layers: int = 4
    heads: int = 12
    kv_heads: int = 4
    dim: int = 128
    hidden: int = 6144
    page: int = 64
    eps: float = 1e-6

    def __post_init__(self):
        if self.heads % self.kv_heads:
            raise ValueError(f"{self.heads} query heads over {self.kv_heads} cache heads")
        if min(self.c_latent, self.width, self.layers, self.hidden) < 1:
            raise ValueError("sizes must be at least 1")

    @property
    def qkv(self) -> int:
        return (self.heads + 2 * self.kv_heads) * self.dim


def random_weights(cfg: Config, seed: int = 0, device="cuda") -> Dict[str, torch.Tensor]:
    """Float weights by name, as a checkpoint would hold them: products
    [out, in], norms [width]."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def product(out, inp, gain=1.0):
        return torch.randn((out, inp), generator=g, device=device) * (gain / math.sqrt(inp))

    w = {"in": product(cfg.width, cfg.c_latent), "out": product(cfg.c_latent, cfg.width),
         "norm": 1 + 0.1 * torch.randn(cfg.width, generator=g, device=device),
         "out_bias": 0.1 * torch.randn(cfg.c_latent, generator=g, device=device)}
    for i in range(cfg.layers):
        w[f"{i}.norm1"] = 1 + 0.1 * torch.randn(cfg.width, generator=g, device=device)
        w[f"{i}.norm2"] = 1 + 0.1 * torch.randn(cfg.width, generator=g, device=device)
        w[f"{i}.qkv"] = product(cfg.qkv, cfg.width)
        w[f"{i}.o"] = product(cfg.width, cfg.heads * cfg.dim, 0.5)
        w[f"{i}.up"] = product(cfg.hidden, cfg.width)
        w[f"{i}.down"] = product(cfg.width, cfg.hidden, 0.5)
    return w


def positions(count: int, width: int, device="cuda") -> torch.Tensor:
    """[count, width] sinusoids, added to the embedded frames."""
    at = torch.arange(count, device=device, dtype=torch.float32)[:, None]
    rate = torch.exp(torch.arange(0, width, 2, device=device, dtype=torch.float32)
                     * (-math.log(10000.0) / width))
    out = torch.empty((count, width), device=device)
    out[:, 0::2] = torch.sin(at * rate)
    out[:, 1::2] = torch.cos(at * rate[: width // 2])
    return out


class LatentGenerator:
    """`streams` sequences of latent frames, each up to max_frames long."""

    def __init__(self, cfg: Config, weights: Dict[str, torch.Tensor], streams: int,
                 max_frames: int):
        self.cfg, self.streams, self.max_frames = cfg, streams, max_frames
        dev = weights["in"].device
        # products in 8 bits with a scale for each output, laid out once
        self.w = {k: avae.quant_q8(v.float().contiguous()) if v.dim() == 2 else v.float()
                  for k, v in weights.items()}
        self.pos = positions(max_frames, cfg.width, dev).bfloat16()
        pages = -(-max_frames // cfg.page)
        self.caches = [avae.KvCacheQ8.empty(streams * pages, cfg.kv_heads, cfg.page, cfg.dim, dev)
                       for _ in range(cfg.layers)]
        self.table = torch.arange(streams * pages, dtype=torch.int32, device=dev).view(streams, pages)
        self.lens = torch.zeros(streams, dtype=torch.int32, device=dev)
        self.one_each = torch.arange(streams + 1, dtype=torch.int32, device=dev)
        self.longest = 0
        self.empty = True

    def _linear(self, q, scale, name, **kw):
        w, w_scale = self.w[name]
        return avae.linear_q8(q, scale, w, w_scale, **kw)

    def _forward(self, frames, cu, most: int):
        """frames [rows, c_latent] float32, the streams' last ones as cu says
        (self.lens counts them already) -> [rows, c_latent]."""
        cfg, bf16 = self.cfg, torch.bfloat16
        rows = frames.shape[0]
        stream = torch.searchsorted(cu[1:].long(), torch.arange(rows, device=frames.device), right=True)
        at = self.lens.long()[stream] - cu.long()[stream + 1] + torch.arange(rows, device=frames.device)
        # the embedded frame and its position start the residual stream
        delta = self._linear(*avae.quant_q8(frames), "in", dtype=bf16)
        h = self.pos[at]
        n_q, n_kv = cfg.heads * cfg.dim, cfg.kv_heads * cfg.dim
        for i, cache in enumerate(self.caches):
            q8, s, h = avae.rms_norm_q8(delta, self.w[f"{i}.norm1"], cfg.eps, residual=h)
            qkv = self._linear(q8, s, f"{i}.qkv", dtype=bf16)
            q = qkv[:, :n_q].unflatten(1, (cfg.heads, cfg.dim))
            k = qkv[:, n_q:n_q + n_kv].unflatten(1, (cfg.kv_heads, cfg.dim))
            v = qkv[:, n_q + n_kv:].unflatten(1, (cfg.kv_heads, cfg.dim))
            avae.kv_write_q8(cache, k, v, self.table, cu, self.lens, max_new=most)
            a = avae.attn_q8(q, cache, self.table, cu, self.lens, max_q=most, max_len=self.longest)
            delta = self._linear(*avae.quant_q8(a.flatten(1)), f"{i}.o", dtype=bf16)
            q8, s, h = avae.rms_norm_q8(delta, self.w[f"{i}.norm2"], cfg.eps, residual=h)
            u = self._linear(q8, s, f"{i}.up", act="silu", dtype=bf16)
            delta = self._linear(*avae.quant_q8(u), f"{i}.down", dtype=bf16)
        q8, s, _ = avae.rms_norm_q8(delta, self.w["norm"], cfg.eps, residual=h)
        return self._linear(q8, s, "out", bias=self.w["out_bias"])

    def prefill(self, prompts: Sequence[torch.Tensor]) -> torch.Tensor:
        """One prompt [n, c_latent] a stream (n >= 1) -> the next frame of
        each, [streams, c_latent]."""
        if not self.empty:
            raise ValueError("prompts go into an empty generator")
        if len(prompts) != self.streams or any(
                p.dim() != 2 or p.shape[0] < 1 or p.shape[1] != self.cfg.c_latent for p in prompts):
            raise ValueError(f"expected {self.streams} prompts [n, {self.cfg.c_latent}]")
        counts = [p.shape[0] for p in prompts]
        if max(counts) > self.max_frames:
            raise ValueError(f"a prompt of {max(counts)} frames: at most {self.max_frames}")
        dev = self.lens.device
        cu = torch.tensor([0] + counts, dtype=torch.int32, device=dev).cumsum(0).int()
        self.lens.copy_(torch.tensor(counts, dtype=torch.int32))
        self.longest, self.empty = max(counts), False
        y = self._forward(torch.cat([p.float() for p in prompts]).to(dev).contiguous(), cu, max(counts))
        return y[cu[1:].long() - 1]

    def step(self, frames: torch.Tensor) -> torch.Tensor:
        """The streams' last frames [streams, c_latent] -> their next ones."""
        if self.empty:
            raise ValueError("a prompt comes first")
        if frames.shape != (self.streams, self.cfg.c_latent):
            raise ValueError(f"expected [{self.streams}, {self.cfg.c_latent}], got {tuple(frames.shape)}")
        if self.longest >= self.max_frames:
            raise ValueError(f"{self.max_frames} frames are written")
        self.lens += 1
        self.longest += 1
        return self._forward(frames.float().contiguous(), self.one_each, 1)

    def generate(self, prompts: Sequence[torch.Tensor], frames: int) -> torch.Tensor:
        """`frames` new frames of each stream after its prompt -> latent
        [streams, c_latent, frames], as the decoder takes it."""
        if frames < 1:
            raise ValueError(f"frames must be at least 1, got {frames}")
        out: List[torch.Tensor] = [self.prefill(prompts)]
        while len(out) < frames:
            out.append(self.step(out[-1]))
        return torch.stack(out, 2).contiguous()


def main():
    import time

    import numpy as np

    from . import workloads as W
    cfg = Config()
    streams, prompt, frames = 2, 40, 400
    gen = LatentGenerator(cfg, random_weights(cfg), streams, prompt + frames)
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [torch.randn((prompt, cfg.c_latent), generator=g, device="cuda") for _ in range(streams)]
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    latent = gen.generate(prompts, frames)
    torch.cuda.synchronize()
    t1 = time.perf_counter()
    dec = avae.Decoder(W.H3, {k: torch.from_numpy(np.ascontiguousarray(v)).cuda()
                              for k, v in W.decoder_tensors(W.H3, 4).items()})
    dec.decode(latent)
    torch.cuda.synchronize()
    t2 = time.perf_counter()
    wave = dec.decode(latent)
    torch.cuda.synchronize()
    t3 = time.perf_counter()
    print(f"{streams} streams x {frames} frames in {1e3 * (t1 - t0):.1f} ms "
          f"({1e3 * (t1 - t0) / frames:.3f} ms a frame), decoded to {tuple(wave.shape)} in "
          f"{1e3 * (t3 - t2):.1f} ms; all finite: {bool(torch.isfinite(wave).all())}")


if __name__ == "__main__":
    main()
