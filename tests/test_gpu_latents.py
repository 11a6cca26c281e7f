"""The latent generator (latents.py): the 8-bit operators run together, and
their latents through the decoder."""
import math

import pytest

from tests.gpu_util import announce

pytestmark = pytest.mark.gpu


def _config(**kw):
    from bigvgan_waveform_decoder_amd.latents import Config
    return Config(**{**dict(c_latent=32, width=192, layers=2, heads=4, kv_heads=2, dim=64, hidden=384,
                            page=16), **kw})


def _plain(cfg, w, frames, start=0):
    """The same network on one stream in float64 with float weights and no
    8-bit values: [n, c_latent] -> [n, c_latent]."""
    import torch
    from bigvgan_waveform_decoder_amd.latents import positions
    w = {k: v.double() for k, v in w.items()}
    n = frames.shape[0]

    def norm(x, g):
        return x / torch.sqrt((x * x).mean(1, keepdim=True) + cfg.eps) * g

    h = frames.double() @ w["in"].t() + positions(n, cfg.width).double()
    hidden = torch.triu(torch.ones((n, n), dtype=torch.bool, device=h.device), 1)
    for i in range(cfg.layers):
        qkv = norm(h, w[f"{i}.norm1"]) @ w[f"{i}.qkv"].t()
        q, k, v = qkv.split([cfg.heads * cfg.dim, cfg.kv_heads * cfg.dim, cfg.kv_heads * cfg.dim], 1)
        out = []
        for r in range(cfg.heads):
            at = r // (cfg.heads // cfg.kv_heads) * cfg.dim
            s = q[:, r * cfg.dim:(r + 1) * cfg.dim] @ k[:, at:at + cfg.dim].t() / math.sqrt(cfg.dim)
            out.append(torch.softmax(s.masked_fill(hidden, -math.inf), 1) @ v[:, at:at + cfg.dim])
        h = h + torch.cat(out, 1) @ w[f"{i}.o"].t()
        u = norm(h, w[f"{i}.norm2"]) @ w[f"{i}.up"].t()
        h = h + (u * torch.sigmoid(u)) @ w[f"{i}.down"].t()
    return norm(h, w["norm"]) @ w["out"].t() + w["out_bias"]


def test_prompt_and_steps_match_the_float_network():
    """Each 8-bit rounding of rows whose largest value is about 3.5 times
    their spread is an error of 3.5 / 127 / sqrt(12) = 0.8% of the spread;
    with weights rounded as well, seven such pairs a layer and two layers add
    to about 0.011 * sqrt(14) = 4% where none cancels.  Twice that and a
    margin for the values' heavier tails: 10%."""
    import torch
    from bigvgan_waveform_decoder_amd.latents import LatentGenerator, random_weights
    announce("latent generator against float64")
    cfg = _config()
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
        want = _plain(cfg, w, frames[b])[n - 1:n + 9]
        assert float((got[b] - want).norm() / want.norm()) <= 0.1


def test_generate_and_decode():
    import torch
    from bigvgan_waveform_decoder_amd import avae, workloads as W
    from bigvgan_waveform_decoder_amd.latents import LatentGenerator, random_weights
    from tests.gpu_util import cuda_dict
    announce("latent generator into the decoder")
    spec = W.scaled_spec(W.H3, 128)
    cfg = _config(c_latent=spec.c_in, page=16)
    gen = LatentGenerator(cfg, random_weights(cfg, 5), 2, 40)
    g = torch.Generator(device="cuda").manual_seed(7)
    prompts = [torch.randn((n, cfg.c_latent), generator=g, device="cuda") for n in (3, 20)]
    latent = gen.generate(prompts, 12)
    assert latent.shape == (2, spec.c_in, 12) and torch.isfinite(latent).all()
    again = LatentGenerator(cfg, random_weights(cfg, 5), 2, 40).generate(prompts, 12)
    assert torch.equal(latent, again)
    wave = avae.Decoder(spec, cuda_dict(W.decoder_tensors(spec, 4))).decode(latent)
    assert wave.shape == (2, 12 * spec.hop) and torch.isfinite(wave).all()
    assert wave.abs().max() <= 1


def test_generator_refusals():
    import torch
    from bigvgan_waveform_decoder_amd.latents import LatentGenerator, random_weights
    with pytest.raises(ValueError, match="heads"):
        _config(heads=3)
    with pytest.raises(ValueError, match="sizes"):
        _config(layers=0)
    cfg = _config()
    gen = LatentGenerator(cfg, random_weights(cfg), 2, 20)
    one = torch.zeros((2, cfg.c_latent), device="cuda")
    with pytest.raises(ValueError, match="prompt comes first"):
        gen.step(one)
    with pytest.raises(ValueError, match="expected 2 prompts"):
        gen.prefill([one])
    with pytest.raises(ValueError, match="at most 20"):
        gen.prefill([one, torch.zeros((21, cfg.c_latent), device="cuda")])
    gen.prefill([one, torch.zeros((20, cfg.c_latent), device="cuda")])
    with pytest.raises(ValueError, match="empty generator"):
        gen.prefill([one, one])
    with pytest.raises(ValueError, match="frames are written"):
        gen.step(one)


def test_generate_refuses_no_frames():
    """No frame asked for is an error, and leaves the generator empty."""
    import torch
    from bigvgan_waveform_decoder_amd.latents import LatentGenerator, random_weights
    cfg = _config()
    gen = LatentGenerator(cfg, random_weights(cfg), 1, 20)
    one = torch.zeros((1, cfg.c_latent), device="cuda")
    for frames in (0, -3):
        with pytest.raises(ValueError, match="frames must be at least 1"):
            gen.generate([one], frames)
    assert gen.generate([one], 1).shape == (1, cfg.c_latent, 1)
