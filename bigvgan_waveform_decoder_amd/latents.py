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

By its Config a network adds positions to the embedded frames, or turns
queries and keys by them (rot), norms each head (head_norm), caps its scores
(cap), sees a window of the last frames, and of its prompt all (sees_prompt).
Drafted frames are checked at once, as a tree:

    after = gen.check(drafts, parents)     # the next frame after each draft
    gen.keep(paths)                        # goes on from those that are right

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
    rot: int = 0                # dims of a head that positions turn; 0: they are added to the frames
    theta: float = 10000.0
    head_norm: bool = False     # RMS norm of each query and key head
    cap: float = 0.0            # scores become cap * tanh(score / cap); 0: as they are
    window: int = 0             # frames in view; 0: all
    sees_prompt: bool = False   # a prompt sees itself whole, and stays in view of the window

    def __post_init__(self):
        if self.heads % self.kv_heads:
            raise ValueError(f"{self.heads} query heads over {self.kv_heads} cache heads")
        if min(self.c_latent, self.width, self.layers, self.hidden) < 1:
            raise ValueError("sizes must be at least 1")
        if self.rot % 2 or not 0 <= self.rot <= self.dim:
            raise ValueError(f"{self.rot} of {self.dim} dims cannot be turned in pairs")
        if self.window < 0:
            raise ValueError("a window is not negative")

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
        if cfg.head_norm:
            for name in ("q_norm", "k_norm"):
                w[f"{i}.{name}"] = 1 + 0.1 * torch.randn(cfg.dim, generator=g, device=device)
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
        # keys, values and their scales, all layers in one: a page of all of them is one copy
        shape = (cfg.layers, streams * pages, cfg.kv_heads, cfg.page, cfg.dim)
        self.held = (*(torch.zeros(shape, dtype=torch.int8, device=dev) for _ in range(2)),
                     *(torch.zeros(shape[:3], device=dev) for _ in range(2)))
        self.caches = [avae.KvCacheQ8(*(t[i] for t in self.held)) for i in range(cfg.layers)]
        self.table = torch.arange(streams * pages, dtype=torch.int32, device=dev).view(streams, pages)
        self.lens = torch.zeros(streams, dtype=torch.int32, device=dev)
        self.one_each = torch.arange(streams + 1, dtype=torch.int32, device=dev)
        self.counts = [0] * streams  # what lens holds, on the host (or what bounds it)
        self.empty = True
        self.rope = avae.Rope.of(cfg.rot, theta=cfg.theta, device=dev) if cfg.rot else None
        self.prompt = torch.zeros(streams, dtype=torch.int32, device=dev)
        self.longest_prompt = 0
        self.drafts = None  # what keep() needs of the last check(): parents, keys and values a layer

    @property
    def longest(self) -> int:
        """The most frames that a stream has; set by who sets `lens` back."""
        return max(self.counts)

    @longest.setter
    def longest(self, frames: int) -> None:
        self.counts = [frames] * self.streams  # (at most: lens has each stream's)

    def _linear(self, q, scale, name, **kw):
        w, w_scale = self.w[name]
        return avae.linear_q8(q, scale, w, w_scale, **kw)

    def _attend(self, q, cache, cu, lens, most: int, longest: int, tree):
        cfg = self.cfg
        args = (q, cache, self.table, cu, lens)
        if tree is not None:
            return avae.attn_tree_q8(*args, tree, max_q=most, max_len=longest, cap=cfg.cap)
        if not cfg.cap and not cfg.sees_prompt:
            return avae.attn_q8(*args, max_q=most, max_len=longest, window=cfg.window)
        return avae.attn_rules_q8(*args, max_q=most, max_len=longest, window=cfg.window, cap=cfg.cap,
                                  prefix=self.prompt if cfg.sees_prompt else None,
                                  max_prefix=self.longest_prompt)

    def _write(self, i: int, k, v, cu, lens, most: int, positions=None):
        """Keys and values of layer i into its cache."""
        if self.rope is None and not self.cfg.head_norm:
            avae.kv_write_q8(self.caches[i], k, v, self.table, cu, lens, max_new=most)
        else:
            avae.kv_write_rope_q8(self.caches[i], k, v, self.table, cu, lens, self.rope,
                                  k_weight=self.w.get(f"{i}.k_norm"), eps=self.cfg.eps,
                                  positions=positions, max_new=most)

    def _tails(self):
        """The page of each stream that its next frame goes into (its last
        one where all are full), and what the caches hold there."""
        col = (self.lens.long() // self.cfg.page).clamp(max=self.table.shape[1] - 1)
        pages = self.table.long().gather(1, col[:, None])[:, 0]
        return pages, [t[:, pages] for t in self.held]

    def _forward(self, frames, cu, lens, most: int, longest: int, tree=None, positions=None):
        """frames [rows, c_latent] float32, the streams' last ones as cu and
        lens say (at their places, or drafts at `positions` that see each other
        by `tree`) -> [rows, c_latent], and the drafts' keys and values a layer
        (none without `tree`)."""
        cfg, bf16 = self.cfg, torch.bfloat16
        rows = frames.shape[0]
        at = positions
        if at is None:
            row = torch.arange(rows, device=frames.device)
            stream = torch.searchsorted(cu[1:].long(), row, right=True)
            at = lens.long()[stream] - cu.long()[stream + 1] + row
        # the embedded frame and its position start the residual stream
        delta = self._linear(*avae.quant_q8(frames), "in", dtype=bf16)
        h = self.pos[at.long()] if not cfg.rot else torch.zeros_like(delta)
        kept = []
        n_q, n_kv = cfg.heads * cfg.dim, cfg.kv_heads * cfg.dim
        for i, cache in enumerate(self.caches):
            q8, s, h = avae.rms_norm_q8(delta, self.w[f"{i}.norm1"], cfg.eps, residual=h)
            qkv = self._linear(q8, s, f"{i}.qkv", dtype=bf16)
            q = qkv[:, :n_q].unflatten(1, (cfg.heads, cfg.dim))
            k = qkv[:, n_q:n_q + n_kv].unflatten(1, (cfg.kv_heads, cfg.dim))
            v = qkv[:, n_q + n_kv:].unflatten(1, (cfg.kv_heads, cfg.dim))
            if self.rope is not None or cfg.head_norm:
                q, _ = avae.qk_norm_rope(q, None, self.rope, self.w.get(f"{i}.q_norm"), eps=cfg.eps,
                                         positions=positions, cu=cu, lens=lens, max_rows=most,
                                         inplace=True)
            self._write(i, k, v, cu, lens, most, positions)
            if tree is not None:
                kept.append((k, v))
            a = self._attend(q, cache, cu, lens, most, longest, tree)
            delta = self._linear(*avae.quant_q8(a.flatten(1)), f"{i}.o", dtype=bf16)
            q8, s, h = avae.rms_norm_q8(delta, self.w[f"{i}.norm2"], cfg.eps, residual=h)
            u = self._linear(q8, s, f"{i}.up", act="silu", dtype=bf16)
            delta = self._linear(*avae.quant_q8(u), f"{i}.down", dtype=bf16)
        q8, s, _ = avae.rms_norm_q8(delta, self.w["norm"], cfg.eps, residual=h)
        return self._linear(q8, s, "out", bias=self.w["out_bias"]), kept

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
        self.counts, self.empty = counts, False
        self.drafts = None
        self.prompt.copy_(self.lens)
        self.longest_prompt = self.longest
        y, _ = self._forward(torch.cat([p.float() for p in prompts]).to(dev).contiguous(), cu, self.lens,
                             max(counts), self.longest)
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
        self.counts = [n + 1 for n in self.counts]
        self.drafts = None
        return self._forward(frames.float().contiguous(), self.one_each, self.lens, 1, self.longest)[0]

    def check(self, drafts: Sequence[torch.Tensor], parents: Sequence[Sequence[int]]) -> List[torch.Tensor]:
        """Drafted frames [n, c_latent] of each stream (n may be 0), draft i
        following draft parents[i] < i of its stream or, with -1, the stream's
        last frame -> the next frame after each draft, [n, c_latent] a stream.
        The streams stay where they are, to the bit: keep() goes on.

        While they are checked the drafts lie in the cache behind their
        stream's frames, in pages of one scale a head: the larger a draft, the
        coarser what shares its page, and one that is not finite makes the
        answers after its stream's drafts so.  The pages that held frames
        before are put back as they were."""
        cfg = self.cfg
        if self.empty:
            raise ValueError("a prompt comes first")
        if cfg.window:
            raise ValueError("drafts are checked without a window")
        if len(drafts) != self.streams or any(
                d.dim() != 2 or d.shape[1] != cfg.c_latent or d.shape[0] != len(p)
                for d, p in zip(drafts, parents)) or len(parents) != self.streams:
            raise ValueError(f"expected {self.streams} drafts [n, {cfg.c_latent}], a parent each")
        if any(not -1 <= p < i for up in parents for i, p in enumerate(up)):
            raise ValueError("a draft's parent comes before it")
        new = [d.shape[0] for d in drafts]
        most, longest = max(new), max(a + b for a, b in zip(self.counts, new))
        if longest > self.max_frames:
            raise ValueError(f"drafts up to frame {longest}: at most {self.max_frames}")
        parents, kept = [list(p) for p in parents], []
        if most == 0:
            y = torch.cat([d.float() for d in drafts])
        else:
            dev = self.lens.device
            cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).int().to(dev)
            lens = self.lens + (cu[1:] - cu[:-1])
            up = torch.tensor([p for u in parents for p in u], dtype=torch.int32, device=dev)
            tree, positions = avae.tree_mask(up, cu, lens, max_rows=most)
            pages, held = self._tails()
            try:
                y, kept = self._forward(torch.cat([d.float() for d in drafts]).to(dev).contiguous(), cu,
                                        lens, most, longest, tree, positions)
            finally:
                for t, was in zip(self.held, held):
                    t[:, pages] = was
        self.drafts = (parents, kept)
        return list(y.split(new))

    def keep(self, paths: Sequence[Sequence[int]]) -> None:
        """Goes on from the last check(): of each stream's drafts those of its
        path, from one that follows the stream down, become its frames (none
        of an empty path)."""
        if self.drafts is None:
            raise ValueError("a check comes first")
        parents, kept = self.drafts
        if len(paths) != self.streams or any(
                not 0 <= i < len(up) or up[i] != before
                for path, up in zip(paths, parents) for before, i in zip([-1, *path], path)):
            raise ValueError("a path goes down through its stream's drafts, each to one that follows it")
        self.drafts = None
        new = [len(p) for p in paths]
        if max(new) == 0:
            return
        dev = self.lens.device
        cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).int().to(dev)
        starts = [sum(len(u) for u in parents[:b]) for b in range(self.streams)]
        rows = torch.tensor([s + i for s, p in zip(starts, paths) for i in p], device=dev)
        self.lens += cu[1:] - cu[:-1]
        self.counts = [a + b for a, b in zip(self.counts, new)]
        for i, (k, v) in enumerate(kept):
            # written anew, one after the other, over what the drafts left
            self._write(i, k[rows], v[rows], cu, self.lens, max(new))

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
