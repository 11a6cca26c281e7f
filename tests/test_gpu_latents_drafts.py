"""What checked drafts leave behind in a latent generator: nothing, unless
they are kept; and what a generator holds."""
import pytest

from tests.gpu_util import announce
from tests.test_gpu_latents_rules import _config

pytestmark = pytest.mark.gpu


def _start(kw, counts=(30, 16, 5, 1), seed=4, frames=80):
    import torch
    from bigvgan_waveform_decoder_amd.latents import LatentGenerator, random_weights
    cfg = _config(**kw)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda n: torch.randn((n, cfg.c_latent), generator=g, device="cuda")
    prompts = [rand(n) for n in counts]
    w = random_weights(cfg, 3)

    def make():
        gen = LatentGenerator(cfg, w, len(counts), frames)
        gen.prefill(prompts)
        return gen
    return make, rand


@pytest.mark.parametrize("what", ["keep", "step", "again"])
@pytest.mark.parametrize("kw", [dict(rot=64, head_norm=True, cap=5.0), dict()], ids=str)
def test_rejected_drafts_leave_nothing(kw, what):
    """Drafts many times as large as the frames, and drafts that are NaN: none
    of them kept, the streams go on to the bit as if nobody had checked."""
    import torch
    announce(f"rejected drafts {kw} {what}")
    make, rand = _start(kw)
    a, b = make(), make()
    parents = [[-1, 0, -1, 1], [-1], [], [-1] + list(range(39))]
    for gain in (1.0, 1000.0, float("nan")):
        after = a.check([rand(len(p)) * gain for p in parents], parents)
        assert [len(x) for x in after] == [len(p) for p in parents]
        if what == "keep":
            a.keep([[]] * 4)
        elif what == "again":
            a.check([rand(1) * 100] * 4, [[-1]] * 4)
        for _ in range(9):  # over a page's end
            frame = rand(4)
            x, y = a.step(frame), b.step(frame)
            assert bool(torch.isfinite(x).all()) and torch.equal(x, y)
        assert a.counts == b.counts and torch.equal(a.lens, b.lens)


def test_kept_drafts_are_written_over_what_was_there():
    """A path kept beside a draft of another range: the streams' pages hold
    what they held, and the path's frames at the range of the two."""
    import torch
    announce("kept drafts beside large ones")
    make, rand = _start(dict(rot=64))
    a = make()
    before = [[t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)] for c in a.caches]
    small = rand(3)
    after = a.check([torch.cat((small[:1], small[1:2] * 1000)), small[2:], small[:0], small[:0]],
                    [[-1, 0], [-1], [], []])
    assert all(bool(torch.isfinite(x).all()) for x in after)
    assert all(torch.equal(t, u) for c, old in zip(a.caches, before)
               for t, u in zip((c.k[:2], c.v[:2], c.k_scale[:2], c.v_scale[:2]), (x[:2] for x in old)))
    a.keep([[0], [0], [], []])
    assert a.counts == [31, 17, 5, 1]
    # the first layer's keys of the kept draft have the range of a frame, not of the large one
    page = a.table[0, 1]
    assert bool((a.caches[0].k_scale[page] <= 4 * before[0][2][page]).all())


def test_a_generator_starts_over():
    """`longest` and `empty` set by a caller, new prompts after that: the same
    bits as from a new generator; drafts of before are forgotten."""
    import torch
    announce("a generator starts over")
    make, rand = _start(dict(rot=64))
    a = make()
    a.check([rand(1)] * 4, [[-1]] * 4)
    for _ in range(20):
        a.step(rand(4))
    a.check([rand(1)] * 4, [[-1]] * 4)
    a.lens.zero_()
    a.longest = 0
    a.empty = True
    assert a.longest == 0
    prompts = [rand(n) for n in (3, 20, 40, 7)]
    x = a.prefill(prompts)
    with pytest.raises(ValueError):
        a.keep([[0]] * 4)  # those were the old streams'
    b = make()
    b.lens.zero_()
    b.longest, b.empty = 0, True
    assert torch.equal(b.prefill(prompts), x)
    frame = rand(4)
    assert torch.equal(a.step(frame), b.step(frame))
    # streams set back: lengths on the device, the longest of them on the host
    a.lens.fill_(3)
    a.longest = 3
    y = a.step(frame)
    assert a.longest == 4 and a.lens.tolist() == [4] * 4 and bool(torch.isfinite(y).all())
    a.check([rand(70)] * 4, [[-1] * 70] * 4)
    with pytest.raises(ValueError):
        a.check([rand(77)] * 4, [[-1] * 77] * 4)


def test_a_prompt_keeps_no_rows():
    """The packed product of a layer is gone when the next one's is made: more
    layers, the same memory beside weights and cache."""
    import torch
    from bigvgan_waveform_decoder_amd.latents import LatentGenerator, random_weights
    announce("memory of a prompt")
    rows, need = 3000, []
    for layers in (2, 8):
        cfg = _config(rot=64, layers=layers)
        gen = LatentGenerator(cfg, random_weights(cfg, 3), 1, rows + 1)
        x = torch.zeros((rows, cfg.c_latent), device="cuda")
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        was = torch.cuda.memory_allocated()
        gen.prefill([x])
        need.append(torch.cuda.max_memory_allocated() - was)
        del gen
    assert need[1] - need[0] < rows * cfg.qkv * 2
