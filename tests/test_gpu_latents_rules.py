"""The latent generator with turned positions, head norms, capped scores, a
prompt in view of a window, and drafts checked as a tree: the operators run
together, against the same network in float64."""
import math

import pytest

from tests.gpu_util import announce

pytestmark = pytest.mark.gpu


def _config(**kw):
    from bigvgan_waveform_decoder_amd.latents import Config
    return Config(**{**dict(c_latent=32, width=192, layers=2, heads=4, kv_heads=2, dim=64, hidden=384,
                            page=16), **kw})


def _plain(cfg, w, frames, prompt, at=None, seen=None):
    """The network on one stream in float64 with float weights and no 8-bit
    values: [n, c_latent] -> [n, c_latent].  at: the frames' positions; seen
    [n, n]: which frames a frame sees (in order, by window and prompt if not
    given)."""
    import torch
    from bigvgan_waveform_decoder_amd.latents import positions
    w = {k: v.double() for k, v in w.items()}
    n, dev = frames.shape[0], frames.device
    at = torch.arange(n, device=dev) if at is None else at
    if seen is None:
        i, j = torch.arange(n, device=dev)[:, None], torch.arange(n, device=dev)
        seen = j <= i
        if cfg.window:
            seen = seen & (j > i - cfg.window)
        if cfg.sees_prompt:
            seen = seen | (j < prompt)

    def norm(x, g):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + cfg.eps) * g

    def turn(x):
        half = cfg.rot // 2
        if not half:
            return x
        f = cfg.theta ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        z = torch.polar(torch.ones(n, half, dtype=torch.float64, device=dev), at.double()[:, None] * f)
        z = z * torch.complex(x[:, :half].contiguous(), x[:, half:2 * half].contiguous())
        return torch.cat((z.real, z.imag, x[:, 2 * half:]), 1)

    h = frames.double() @ w["in"].t()
    if not cfg.rot:
        h = h + positions(int(at.max()) + 1, cfg.width, dev).double()[at]
    for i in range(cfg.layers):
        qkv = norm(h, w[f"{i}.norm1"]) @ w[f"{i}.qkv"].t()
        q, k, v = (x.unflatten(1, (-1, cfg.dim)) for x in qkv.split(
            [cfg.heads * cfg.dim, cfg.kv_heads * cfg.dim, cfg.kv_heads * cfg.dim], 1))
        if cfg.head_norm:
            q, k = norm(q, w[f"{i}.q_norm"]), norm(k, w[f"{i}.k_norm"])
        out = []
        for r in range(cfg.heads):
            g = r // (cfg.heads // cfg.kv_heads)
            s = turn(q[:, r]) @ turn(k[:, g]).t() / math.sqrt(cfg.dim)
            if cfg.cap:
                s = cfg.cap * torch.tanh(s / cfg.cap)
            out.append(torch.softmax(s.masked_fill(~seen, -math.inf), 1) @ v[:, g])
        h = h + torch.cat(out, 1) @ w[f"{i}.o"].t()
        u = norm(h, w[f"{i}.norm2"]) @ w[f"{i}.up"].t()
        h = h + (u * torch.sigmoid(u)) @ w[f"{i}.down"].t()
    return norm(h, w["norm"]) @ w["out"].t() + w["out_bias"]


CONFIGS = [dict(rot=64), dict(rot=26, head_norm=True), dict(rot=64, head_norm=True, cap=5.0),
           dict(rot=32, cap=3.0, window=11, sees_prompt=True), dict(window=20),
           dict(head_norm=True, sees_prompt=True)]


@pytest.mark.parametrize("kw", CONFIGS, ids=str)
def test_prompt_and_steps_match_the_float_network(kw):
    """Each 8-bit rounding of rows whose largest value is about 3.5 times
    their spread is an error of 3.5 / 127 / sqrt(12) = 0.8% of the spread;
    with weights rounded as well, seven such pairs a layer and two layers add
    to about 0.011 * sqrt(14) = 4% where none cancels.  Twice that and a
    margin for the values' heavier tails: 10%."""
    import torch
    from bigvgan_waveform_decoder_amd.latents import LatentGenerator, random_weights
    announce(f"latent generator {kw} against float64")
    cfg = _config(**kw)
    w = random_weights(cfg, 3)
    g = torch.Generator(device="cuda").manual_seed(2)
    counts = [37, 5]
    frames = [torch.randn((n + 9, cfg.c_latent), generator=g, device="cuda") for n in counts]
    gen = LatentGenerator(cfg, w, 2, 64)
    got = [gen.prefill([f[:n] for f, n in zip(frames, counts)])]
    for t in range(9):  # the streams' frames are given, not the generator's own
        got.append(gen.step(torch.stack([f[n + t] for f, n in zip(frames, counts)])))
    got = torch.stack(got, 1).double()
    for b, n in enumerate(counts):
        want = _plain(cfg, w, frames[b], n)[n - 1:n + 9]
        assert float((got[b] - want).norm() / want.norm()) <= 0.1


@pytest.mark.parametrize("kw", [dict(rot=64), dict(rot=64, head_norm=True, cap=5.0), dict()], ids=str)
def test_drafts_are_checked_and_kept(kw):
    """A tree of drafts, a path of them kept, frames after that: each the
    float network's on the frames that it follows (tolerance as above)."""
    import torch
    from bigvgan_waveform_decoder_amd.latents import LatentGenerator, random_weights
    announce(f"drafts {kw}")
    cfg = _config(**kw)
    w = random_weights(cfg, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda n: torch.randn((n, cfg.c_latent), generator=g, device="cuda")
    prompts = [rand(30), rand(14), rand(3)]
    gen = LatentGenerator(cfg, w, 3, 64)
    gen.prefill(prompts)
    past = [p for p in prompts]
    for parents, paths in (([[-1, 0, 0, 1, -1, 4, 3], [-1], []], [[0, 1, 3], [], []]),
                           ([[-1, -1], [-1, 0, 1, 2], [-1, 0, 0]], [[1], [0, 1, 2, 3], [0, 2]])):
        drafts = [rand(len(p)) for p in parents]
        after = gen.check(drafts, parents)
        for b, (d, up) in enumerate(zip(drafts, parents)):
            assert after[b].shape == d.shape
            want = []
            for i in range(len(up)):
                line = [i]
                while up[line[0]] >= 0:
                    line.insert(0, up[line[0]])
                want.append(_plain(cfg, w, torch.cat((past[b], d[line])), len(prompts[b]))[-1])
            if up:
                want = torch.stack(want)
                assert float((after[b].double() - want).norm() / want.norm()) <= 0.1
        gen.keep(paths)
        past = [torch.cat((p, d[path])) for p, d, path in zip(past, drafts, paths)]
        assert gen.lens.tolist() == [len(p) for p in past] == gen.counts
        frame = rand(3)
        got = gen.step(frame)
        past = [torch.cat((p, f[None])) for p, f in zip(past, frame)]
        for b in range(3):
            want = _plain(cfg, w, past[b], len(prompts[b]))[-1]
            assert float((got[b].double() - want).norm() / want.norm()) <= 0.1


def test_refusals_of_drafts():
    import torch
    from bigvgan_waveform_decoder_amd.latents import LatentGenerator, random_weights
    announce("drafts refused")
    cfg = _config(rot=64)
    w = random_weights(cfg, 3)
    x = torch.zeros((2, cfg.c_latent), device="cuda")
    gen = LatentGenerator(cfg, w, 1, 8)
    with pytest.raises(ValueError):
        gen.check([x], [[-1, 0]])  # no prompt yet
    gen.prefill([x])
    for drafts, parents in (([x], [[-1]]), ([x], [[0, 0]]), ([x], [[-1, 1]]), ([x], [[-1, -2]]), ([x, x], [[-1, 0]]),
                            ([torch.zeros((7, cfg.c_latent), device="cuda")], [list(range(-1, 6))])):
        with pytest.raises(ValueError):
            gen.check(drafts, parents)
    with pytest.raises(ValueError):
        gen.keep([[]])  # nothing checked
    gen.check([x], [[-1, -1]])
    for paths in ([[0, 1]], [[2]], [[1, 0]], [[-1]], [[], []]):
        with pytest.raises(ValueError):
            gen.keep(paths)
    gen.keep([[1]])
    assert gen.counts == [3]
    with pytest.raises(ValueError):
        gen.keep([[0]])
    with pytest.raises(ValueError):
        LatentGenerator(_config(window=4), w, 1, 8).check([x], [[-1, 0]])
    for bad in (dict(rot=3), dict(rot=66), dict(rot=-2), dict(window=-1)):
        with pytest.raises(ValueError):
            _config(**bad)
