"""Positions and masks of the latent generator's attention, as cases that can be timed and checked.

Generators whose attention turns queries and keys by their position, norms them for each head, caps the scores, lets distance weigh,
keeps a conditioning prompt in view, or checks a tree of drafted frames at once need these beside the 8-bit norm, product, cache and
attention.  `run` computes one of them, in elementary torch operations where `own` is false and through the library's entry points
where it is true.

Kinds of cases and what they return:
  turn    queries and keys, normed for each head and turned by their positions
  append  keys (normed, turned) and values of every page that the new tokens went into, read back after the write
  rules   the attention's output rows (and the log sums), scores capped, biased by distance, a prefix in view of all rows
  tree    the same for rows that are a tree of drafts (and the drafts' positions, where the tree comes as parents)
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
# what the cache is read back in: a value beside the border of two 8-bit steps may fall to either side of it
BACK = {"f32": torch.float16, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated frame of one stream, after a minute
        dict(name="turn-step", kind="turn", seqs=1, new_lo=1, new_hi=1, past_hi=2400, heads=12, kv_heads=4, dim=128, rot=128, pairs="halves", norm=True, stretch=1.0, dtype="bf16"),
        # four prompts of a minute or two for a generator stretched to eight times its trained length
        dict(name="turn-prompt", kind="turn", seqs=4, new_lo=2000, new_hi=6000, past_hi=20000, heads=12, kv_heads=4, dim=128, rot=128, pairs="halves", norm=True, stretch=8.0, dtype="bf16"),
        # neighbouring dims as pairs, an odd part of the head, far positions, no norm, in float32
        dict(name="turn-odd", kind="turn", seqs=3, new_lo=601, new_hi=803, past_hi=900000, heads=16, kv_heads=2, dim=64, rot=50, pairs="neighbours", norm=False, stretch=1.0, dtype="f32"),
        # 64 streams append one frame each, most of them into pages that hold frames already
        dict(name="append-step", kind="append", seqs=64, new_lo=1, new_hi=1, past_hi=2400, kv_heads=4, dim=128, page=64, rot=128, pairs="halves", norm=True, stretch=1.0, tree=False, dtype="bf16"),
        # three ragged prompts are written, one of them after a past
        dict(name="append-prompt", kind="append", seqs=3, new_lo=2000, new_hi=6000, past_hi=700, kv_heads=16, dim=64, page=32, rot=64, pairs="neighbours", norm=False, stretch=1.0, tree=False, dtype="f32"),
        # trees of drafts: several tokens at one position, half of the head turned, small pages
        dict(name="append-drafts", kind="append", seqs=16, new_lo=5, new_hi=24, past_hi=4000, kv_heads=4, dim=128, page=16, rot=64, pairs="halves", norm=True, stretch=4.0, tree=True, dtype="f16"),
        # one stream's next frame after a minute, scores capped and weighed by distance
        dict(name="rules-step", kind="rules", seqs=1, q_lo=1, q_hi=1, past_lo=2399, past_hi=2399, heads=12, kv_heads=4, dim=128, page=64, window=0, cap=30.0, bias=True, prefix=0, lse=False, dtype="bf16"),
        # two prompts whose conditioning part sees itself whole, scores capped
        dict(name="rules-prompt", kind="rules", seqs=2, q_lo=3500, q_hi=4000, past_lo=0, past_hi=3000, heads=12, kv_heads=12, dim=128, page=64, window=0, cap=50.0, bias=False, prefix=1500, lse=False, dtype="bf16"),
        # 48 streams of up to ten minutes, a frame each: the last minute and the conditioning part in view
        dict(name="rules-stream", kind="rules", seqs=48, q_lo=1, q_hi=1, past_lo=200, past_hi=24000, heads=16, kv_heads=2, dim=64, page=16, window=2401, cap=0.0, bias=True, prefix=333, lse=True, dtype="f32"),
        # a tree of drafts for one stream
        dict(name="tree-step", kind="tree", seqs=1, q_lo=24, q_hi=24, past_lo=2399, past_hi=2399, heads=12, kv_heads=4, dim=128, page=64, cap=0.0, parents=False, lse=False, dtype="bf16"),
        # trees for 16 streams of up to ten minutes
        dict(name="tree-batch", kind="tree", seqs=16, q_lo=33, q_hi=64, past_lo=500, past_hi=24000, heads=12, kv_heads=4, dim=128, page=64, cap=0.0, parents=False, lse=False, dtype="bf16"),
        # small trees of several sizes in float32, given as parents, scores capped
        dict(name="tree-small", kind="tree", seqs=7, q_lo=1, q_hi=13, past_lo=100, past_hi=1900, heads=16, kv_heads=2, dim=64, page=16, cap=20.0, parents=True, lse=True, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    kind = rng.choice(["turn", "append", "rules", "tree"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    kv_heads, dim, page = rng.choice([1, 2, 4, 8, 12]), rng.choice([64, 64, 128, 128, 128, 256]), rng.choice([16, 32, 64, 128])
    group = rng.choice([1, 2, 3, 4, 8])
    case = dict(kind=kind, seqs=_log(rng, 1, 64))
    if kind in ("turn", "append"):
        if kind == "turn":
            dim = rng.choice([dim, dim, 80, 96])
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)])
        hi = 1 if rng.random() < 0.4 else _log(rng, 2, 6000)
        past = _log(rng, 1, 900000 if kind == "turn" else 5000)
        case.update(new_lo=max(1, hi // 3), new_hi=hi, past_hi=past)
        if kind == "turn":
            case.update(heads=kv_heads * group, kv_heads=kv_heads, dim=dim)
        else:
            case.update(kv_heads=kv_heads, dim=dim, page=page)
        case.update(rot=rot, pairs=rng.choice(["halves", "neighbours"]), norm=rng.random() < 0.6, stretch=rng.choice([1.0, 1.0, 4.0, 8.0]))
        if kind == "append":
            case.update(tree=hi <= 64 and rng.random() < 0.5)
        return dict(case, dtype=dtype)
    hi = 1 if rng.random() < 0.4 else _log(rng, 2, 4000 if kind == "rules" else 64)
    past = _log(rng, 16, 24000)
    case.update(q_lo=max(1, hi // 2), q_hi=hi, past_lo=past // rng.choice([1, 2, 20]), past_hi=past, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page)
    cap = rng.choice([0.0, 0.0, 15.0, 50.0])
    if kind == "rules":
        # at least one of the rules
        bias = rng.random() < 0.5
        prefix = rng.choice([0, _log(rng, 1, 2000)]) if bias or cap else _log(rng, 1, 2000)
        return dict(case, window=rng.choice([0, 0, _log(rng, 32, 2500)]), cap=cap, bias=bias, prefix=prefix, lse=rng.random() < 0.3, dtype=dtype)
    return dict(case, cap=cap, parents=rng.random() < 0.5, lse=rng.random() < 0.3, dtype=dtype)


def draw(rng):
    """A case of the same ranges that asks for no more than the largest listed one of its kind."""
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["kind"], (0.0, 0.0))
        most[c["kind"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    while True:
        c = _drawn(rng)
        w = work(c)
        b, f = most[c["kind"]]
        if w["bytes"] <= b and w["flops"] <= f and _padded(c) <= 2e9:
            return c


def _padded(case):
    """Values of the largest array that the plain form of an attention makes."""
    if "q_hi" not in case:
        return 0.0
    new, total = _lengths(case)
    return float(case["seqs"]) * max(total) * max(case["heads"] * max(new), case["kv_heads"] * case["dim"])


def _random(case):
    return random.Random("%d %d %d" % (case["seqs"], case["past_hi"], case["dim"]))


def _lengths(case):
    """New tokens and length afterwards of each sequence: by the case alone, so that what it asks for is known."""
    r = _random(case)
    lo, hi = (case["q_lo"], case["q_hi"]) if "q_hi" in case else (case["new_lo"], case["new_hi"])
    new = [r.randint(lo, hi) for _ in range(case["seqs"])]
    past = [r.randint(case.get("past_lo", 0), case["past_hi"]) for _ in range(case["seqs"])]
    return new, [a + b for a, b in zip(new, past)]


def _prefixes(case):
    """Tokens of each sequence's conditioning part."""
    r = _random(case)
    return [r.randint(case["prefix"] // 2, case["prefix"]) for _ in range(case["seqs"])]


def _parents(case):
    """The parent of each draft among its sequence's drafts, -1 for those that follow the last token."""
    r, out = _random(case), []
    for n in _lengths(case)[0]:
        out += [-1] + [r.randint(max(-1, i - 6), i - 1) for i in range(1, n)]
    return out


def _lineage(case):
    """Of each draft the drafts that it follows, itself the last: places in its sequence."""
    parents, out, at = _parents(case), [], 0
    for n in _lengths(case)[0]:
        for i in range(n):
            p = parents[at + i]
            out.append(([] if p < 0 else out[at + p]) + [i])
        at += n
    return out


def work(case):
    es = SIZE[case["dtype"]]
    new, total = _lengths(case)
    row = case["kv_heads"] * case["dim"]
    if case["kind"] == "turn":
        return {"bytes": 2 * sum(new) * (case["heads"] + case["kv_heads"]) * case["dim"] * es, "flops": 0}
    if case["kind"] == "append":
        back = sum(t - (t - n) // case["page"] * case["page"] for n, t in zip(new, total))
        # new rows in, their 8-bit values out, and the touched pages' rows out once more as the values they stand for
        return {"bytes": 2 * row * (sum(new) * (es + 1) + back * (1 + 2)), "flops": 0}
    pairs = keys = 0
    if case["kind"] == "tree":
        pairs = sum((t - n) * n for n, t in zip(new, total)) + sum(len(x) for x in _lineage(case))
        keys = sum(total)
    else:
        w = case["window"]
        for n, t, c in zip(new, total, _prefixes(case)):
            for p in range(t - n, t):
                lo, c1 = (max(0, p - w + 1) if w else 0), min(c, t)
                pairs += max(c1, p + 1) - lo + min(lo, c1)
            lo = max(0, t - n - w + 1) if w else 0
            keys += t - lo + min(lo, c)
    return {"bytes": 2 * row * keys + 2 * sum(new) * case["heads"] * case["dim"] * es, "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _offsets(counts):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _turning(s, g):
    """What turns the heads: frequencies (slow ones stretched for long contexts), their gain, the norms' weights."""
    half = s["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    s["amp"] = 1.0
    if s["stretch"] > 1:
        turns = freq * (4096 / (2 * math.pi))
        keep = ((turns - 1) / 31).clamp(0, 1)
        freq = freq * keep + freq / s["stretch"] * (1 - keep)
        s["amp"] = 0.1 * math.log(s["stretch"]) + 1
    s["freq"] = freq.float().cuda()
    s["wq"] = 1 + 0.2 * _normal(g, s["dim"]) if s["norm"] else None
    s["wk"] = 1 + 0.2 * _normal(g, s["dim"]) if s["norm"] else None


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    new, total = _lengths(case)
    s["cu"], s["lens"] = _offsets(new), torch.tensor(total, dtype=torch.int32, device="cuda")
    s["total"], s["max_new"], s["max_len"] = sum(new), max(new), max(total)
    b, h, d = case["seqs"], case["kv_heads"], case["dim"]
    if case["kind"] == "turn":
        _turning(s, g)
        # queries and keys lie beside the values in the rows of one product
        qkv = (_normal(g, s["total"], case["heads"] + 2 * h, d) * torch.exp(0.5 * _normal(g, d))).to(dt)
        s["q"], s["k"] = qkv[:, : case["heads"]], qkv[:, case["heads"] : case["heads"] + h]
        return s
    p = case["page"]
    pages = [-(-t // p) for t in total]
    count = sum(pages) + 3  # a few pages belong to nobody
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)[: sum(pages)].cpu()
    table = torch.full((b, max(pages)), -1, dtype=torch.int32)
    at = 0
    for i, c in enumerate(pages):
        table[i, :c] = order[at : at + c]
        at += c
    s["table"] = table.cuda()
    # keys have a few large channels; every page and head has its own range
    wide = torch.exp(0.8 * _normal(g, h, 1, d))
    for name, by in (("k", wide), ("v", 1.0)):
        q8, scales = [], []
        for at in range(0, count, 4096):
            x = _normal(g, min(4096, count - at), h, p, d) * by
            sc = x.abs().amax((2, 3)) / 127
            q8.append((x / sc[:, :, None, None]).round().to(torch.int8))
            scales.append(sc)
        s[name + "8"], s[name + "s"] = torch.cat(q8), torch.cat(scales)
    if case["kind"] == "append":
        _turning(s, g)
        s["k"] = (_normal(g, s["total"], h, d) * wide[:, 0]).to(dt)
        s["v"] = _normal(g, s["total"], h, d).to(dt)
        s["pos"] = None
        if case["tree"]:
            depth = torch.tensor([len(x) - 1 for x in _lineage(case)], dtype=torch.int32)
            start = torch.tensor([t - n for n, t in zip(new, total)], dtype=torch.int32)
            s["pos"] = (depth + start.repeat_interleave(torch.tensor(new))).cuda()
        # every token of the pages that the new ones go into is read back
        back = [t - (t - n) // p * p for n, t in zip(new, total)]
        s["back"], s["back_total"], s["max_back"] = _offsets(back), sum(back), max(back)
        return s
    # scores as large as a cap is there for
    s["q"] = (_normal(g, s["total"], case["heads"], d) * (4 if case["cap"] else 1)).to(dt)
    if case["kind"] == "rules":
        heads = torch.arange(1, case["heads"] + 1, device="cuda", dtype=torch.float32)
        s["slopes"] = torch.exp2(-8 * heads / case["heads"]) if case["bias"] else None
        s["pre"] = torch.tensor(_prefixes(case), dtype=torch.int32, device="cuda") if case["prefix"] else None
        return s
    s["up"] = torch.tensor(_parents(case), dtype=torch.int32, device="cuda")
    words = -(-max(new) // 32)
    bits = torch.zeros((s["total"], words), dtype=torch.int64)
    for i, line in enumerate(_lineage(case)):
        for j in line:
            bits[i, j // 32] += 1 << (j % 32)
    s["seen"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32).cuda()
    return s


# ------------------------------------------------------------------ plain forms

def _places(s, cu, total):
    """Sequence and position of each packed token: a sequence's tokens are its last ones."""
    tok = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu[1:].long(), tok, right=True)
    pos = s["lens"].long()[seq] - cu.long()[seq + 1] + tok
    return seq, pos


def _turn(s, x, weight, pos):
    """Heads x [tokens, heads, dim] normed and turned, in float32."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(2, keepdim=True) + EPS) * weight
    angle = pos.double()[:, None] * s["freq"].double()
    cos, sin = (torch.cos(angle) * s["amp"]).float()[:, None], (torch.sin(angle) * s["amp"]).float()[:, None]
    rot = s["rot"]
    out = x.clone()
    if s["pairs"] == "halves":
        a, b = x[:, :, : rot // 2], x[:, :, rot // 2 : rot]
        out[:, :, : rot // 2] = a * cos - b * sin
        out[:, :, rot // 2 : rot] = b * cos + a * sin
    else:
        a, b = x[:, :, 0:rot:2], x[:, :, 1:rot:2]
        out[:, :, 0:rot:2] = a * cos - b * sin
        out[:, :, 1:rot:2] = b * cos + a * sin
    return out


def _plain_turn(s):
    dt = DTYPES[s["dtype"]]
    pos = _places(s, s["cu"], s["total"])[1]
    return {"q": _turn(s, s["q"], s["wq"], pos).to(dt), "k": _turn(s, s["k"], s["wk"], pos).to(dt)}


def _plain_write(s, x, q8, scales):
    p = s["page"]
    seq, pos = _places(s, s["cu"], s["total"])
    page, slot = s["table"].long()[seq, pos // p], pos % p
    # the range of each page: of its new tokens, and of those it held before
    amax = torch.zeros_like(scales).scatter_reduce_(0, page[:, None].expand(-1, s["kv_heads"]), x.abs().amax(2), "amax")
    start = s["lens"].long() - (s["cu"][1:] - s["cu"][:-1]).long()
    at = s["table"].long().gather(1, (start // p).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0]
    held = torch.arange(p, device="cuda") < (start % p)[:, None]
    old = torch.where((start % p > 0)[:, None], scales[at], 0.0)
    new = amax / 127
    new[at] = torch.maximum(new[at], old)
    # tokens that a page held are moved to its new range
    before = q8[at]
    moved = (before.float() * old[:, :, None, None] / new[at][:, :, None, None]).round().to(torch.int8)
    grown = held[:, None, :, None] & (new[at] > old)[:, :, None, None]
    q8[at] = torch.where(grown, moved, before)
    touched = torch.cat((page, at))
    scales[touched] = new[touched]
    by = new[page][:, :, None]
    q8[page, :, slot] = torch.where(by > 0, (x / by).round(), 0.0).clamp(-127, 127).to(torch.int8)


def _plain_read(s, q8, scales):
    seq, pos = _places(s, s["back"], s["back_total"])
    page = s["table"].long()[seq, pos // s["page"]]
    return (q8[page, :, pos % s["page"]].float() * scales[page][:, :, None]).to(BACK[s["dtype"]])


def _plain_append(s):
    pos = s["pos"] if s["pos"] is not None else _places(s, s["cu"], s["total"])[1]
    _plain_write(s, _turn(s, s["k"], s["wk"], pos), s["k8"], s["ks"])
    _plain_write(s, s["v"].float(), s["v8"], s["vs"])
    return {"k": _plain_read(s, s["k8"], s["ks"]), "v": _plain_read(s, s["v8"], s["vs"])}


def _plain_lineage(s):
    """seen [tokens, drafts of a sequence] and the drafts' depths, from their parents."""
    b, n = s["seqs"], s["max_new"]
    seq, _ = _places(s, s["cu"], s["total"])
    row = torch.arange(s["total"], device="cuda") - s["cu"].long()[seq]
    reach = torch.eye(n, device="cuda").repeat(b, 1, 1)
    follows = s["up"] >= 0
    reach[seq[follows], row[follows], s["up"].long()[follows]] = 1
    for _ in range(max(1, (n - 1).bit_length())):
        reach = (torch.matmul(reach, reach) > 0).float()
    seen = reach[seq, row] > 0
    return seen, seen.sum(1) - 1


def _plain_attend(s):
    b, h, d, p = s["seqs"], s["kv_heads"], s["dim"], s["page"]
    group, n = s["heads"] // h, s["max_new"]
    table = s["table"].long().clamp(min=0)
    dt = DTYPES[s["dtype"]]

    def read(q8, scales):  # [sequences, heads, positions, dim]
        x = q8[table].float() * scales[table][..., None, None]
        return x.transpose(1, 2).reshape(b, h, -1, d)

    keys, values = read(s["k8"], s["ks"]), read(s["v8"], s["vs"])
    seq, pos = _places(s, s["cu"], s["total"])
    row = torch.arange(s["total"], device="cuda") - s["cu"].long()[seq]
    q = torch.zeros((b, n, h, group, d), device="cuda")
    q[seq, row] = s["q"].float().view(-1, h, group, d)
    q = q.permute(0, 2, 1, 3, 4).reshape(b, h, n * group, d)
    scores = (q / math.sqrt(d)) @ keys.transpose(2, 3)
    if s["cap"]:
        scores = scores.div_(s["cap"]).tanh_().mul_(s["cap"])
    at = torch.full((b, n), -1, device="cuda")
    at[seq, row] = pos
    key = torch.arange(keys.shape[2], device="cuda")
    outs = {}
    if s["kind"] == "rules":
        seen = key <= at[:, :, None]
        if s["window"]:
            seen &= key > at[:, :, None] - s["window"]
        if s["pre"] is not None:
            seen |= key < torch.minimum(s["pre"], s["lens"])[:, None, None]
        if s["slopes"] is not None:
            far = (key - at[:, :, None]).abs().float()
            view = scores.view(b, h, n, group, -1)
            for i in range(group):  # in turns, for the memory
                view[:, :, :, i] -= s["slopes"].view(h, group)[:, i][:, None, None] * far[:, None]
    else:
        if s["parents"]:
            drafts, depth = _plain_lineage(s)
            outs["pos"] = (s["lens"] - (s["cu"][1:] - s["cu"][:-1]))[seq] + depth.int()
        else:
            j = torch.arange(n, device="cuda")
            drafts = (s["seen"][:, j // 32] >> (j % 32)) & 1 > 0
        start = s["lens"].long() - (s["cu"][1:] - s["cu"][:-1]).long()
        among = key - start[:, None]  # [sequences, keys]: which draft a key is
        mine = torch.zeros((b, n, n), dtype=torch.bool, device="cuda")
        mine[seq, row] = drafts
        here = (among >= 0) & (among < n) & (key < s["lens"][:, None])
        seen = mine.gather(2, among.clamp(0, n - 1)[:, None].expand(-1, n, -1)) & here[:, None]
        seen |= (among < 0)[:, None]
    seen = seen[:, None, :, None].expand(-1, -1, -1, group, -1).reshape(b, 1, n * group, -1)
    scores = scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(3, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    scores = torch.exp_(scores.sub_(top))
    total = scores.sum(3, keepdim=True)
    out = (scores @ values) / torch.where(total > 0, total, 1.0)
    out = out.view(b, h, n, group, d).transpose(1, 2)[seq, row]
    outs["out"] = out.reshape(-1, s["heads"], d).to(dt)
    if s["lse"]:
        lse = (top + torch.log(total)).view(b, h, n, group).transpose(1, 2)[seq, row]
        outs["lse"] = lse.reshape(-1, s["heads"])
    return outs


def _own(s):
    from bigvgan_waveform_decoder_amd import avae

    dt = DTYPES[s["dtype"]]
    if s["kind"] in ("turn", "append"):
        rope = avae.Rope(s["freq"], interleaved=s["pairs"] == "neighbours", amp=s["amp"])
    if s["kind"] == "turn":
        q, k = avae.qk_norm_rope(s["q"], s["k"], rope, q_weight=s["wq"], k_weight=s["wk"], eps=EPS, cu=s["cu"], lens=s["lens"], max_rows=s["max_new"])
        return {"q": q, "k": k}
    cache = avae.KvCacheQ8(s["k8"], s["v8"], s["ks"], s["vs"])
    if s["kind"] == "append":
        avae.kv_write_rope_q8(cache, s["k"], s["v"], s["table"], s["cu"], s["lens"], rope, k_weight=s["wk"], eps=EPS, positions=s["pos"], max_new=s["max_new"])
        k, v = avae.kv_read_q8(cache, s["table"], s["back"], s["lens"], total=s["back_total"], max_rows=s["max_back"], dtype=BACK[s["dtype"]])
        return {"k": k, "v": v}
    outs = {}
    sizes = dict(max_q=s["max_new"], max_len=s["max_len"], cap=s["cap"], return_lse=s["lse"])
    if s["kind"] == "rules":
        got = avae.attn_rules_q8(s["q"], cache, s["table"], s["cu"], s["lens"], window=s["window"], slopes=s["slopes"], prefix=s["pre"], max_prefix=s["prefix"], **sizes)
    else:
        tree = s["seen"]
        if s["parents"]:
            tree, outs["pos"] = avae.tree_mask(s["up"], s["cu"], s["lens"], max_rows=s["max_new"])
        got = avae.attn_tree_q8(s["q"], cache, s["table"], s["cu"], s["lens"], tree, **sizes)
    outs["out"], outs["lse"] = got if s["lse"] else (got, None)
    return {k: v for k, v in outs.items() if v is not None}


def run(state):
    if own:
        return _own(state)
    return {"turn": _plain_turn, "append": _plain_append, "rules": _plain_attend, "tree": _plain_attend}[state["kind"]](state)


# ------------------------------------------------------------------ 64 bits

def _exact_turn(s, x, weight, pos):
    """A complex number for each pair, turned by a unit one."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    rot, half = s["rot"], s["rot"] // 2
    if s["pairs"] == "halves":
        pairs = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous())
    else:
        pairs = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], half, 2).contiguous())
    angle = torch.outer(pos.double(), s["freq"].double())
    pairs = pairs * torch.polar(torch.full_like(angle, s["amp"]), angle)[:, None]
    turned = torch.cat((pairs.real, pairs.imag), -1) if s["pairs"] == "halves" else torch.view_as_real(pairs).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _exact_positions(s):
    new, total = _lengths(s)
    return torch.cat([torch.arange(t - n, t) for n, t in zip(new, total)]).cuda()


def _exact_rows(x, scale):
    """x in 8 bits at a scale that is stored in 32."""
    scale = scale.float().double()
    return torch.round(x / scale).clamp(-127, 127), scale


def _exact_cache(s):
    p, outs = s["page"], {}
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    pos = _exact_positions(s) if s["pos"] is None else s["pos"]
    for name in ("k", "v"):
        x, got = _exact_turn(s, s["k"], s["wk"], pos) if name == "k" else s["v"].double(), []
        for i, t in enumerate(lens):
            n = cu[i + 1] - cu[i]
            for j in range((t - n) // p, -(-t // p)):
                lo, hi = max(t - n, j * p), min(t, (j + 1) * p)
                rows = x[cu[i] + lo - (t - n) : cu[i] + hi - (t - n)].transpose(0, 1)
                scale = (rows.abs().amax((1, 2)) / 127).float()
                held, was = s[name + "8"][table[i][j]], s[name + "s"][table[i][j]]
                held = held[:, : lo - j * p].double()
                if lo > j * p:
                    scale = torch.maximum(scale, was)
                q, by = _exact_rows(rows, scale[:, None, None])
                held = torch.round(held * was.double()[:, None, None] / by)
                got.append((torch.cat((held, q), 1) * by).transpose(0, 1))
        outs[name] = torch.cat(got)
    return outs


def _exact_attend(s):
    d, p, group = s["dim"], s["page"], s["heads"] // s["kv_heads"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    out = torch.zeros((s["total"], s["heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["total"], s["heads"]), dtype=torch.float64, device="cuda")
    lines = _lineage(s) if s["kind"] == "tree" else None
    for i, t in enumerate(lens):
        n = cu[i + 1] - cu[i]
        pages = s["table"][i, : -(-t // p)].long()
        at = torch.arange(t - n, t, device="cuda")[:, None]
        key = torch.arange(t, device="cuda")
        if lines is not None:
            hidden = torch.ones((n, t), dtype=torch.bool)
            hidden[:, : t - n] = False
            for r in range(n):
                hidden[r, [t - n + j for j in lines[cu[i] + r]]] = False
            hidden = hidden.cuda()
        else:
            hidden = key > at
            if s["window"]:
                hidden = hidden | (at - key >= s["window"])
            if s["prefix"]:
                hidden = hidden & (key >= s["pre"][i])
        for h in range(s["kv_heads"]):
            k = (s["k8"][pages, h].double() * s["ks"][pages, h].double()[:, None, None]).reshape(-1, d)[:t]
            v = (s["v8"][pages, h].double() * s["vs"][pages, h].double()[:, None, None]).reshape(-1, d)[:t]
            for r in range(h * group, (h + 1) * group):
                x = torch.mm(s["q"][cu[i] : cu[i + 1], r].double(), k.t()) * d**-0.5
                if s["cap"]:
                    x = s["cap"] * torch.tanh(x / s["cap"])
                if s["kind"] == "rules" and s["bias"]:
                    x = x - s["slopes"][r].double() * (at - key).abs()
                x[hidden] = -math.inf
                out[cu[i] : cu[i + 1], r] = torch.mm(torch.softmax(x, 1), v)
                lse[cu[i] : cu[i + 1], r] = torch.logsumexp(x, 1)
    outs = {"out": out}
    if lines is not None and s["parents"]:
        depth = torch.tensor([len(x) - 1 for x in lines], dtype=torch.int32, device="cuda")
        seq = torch.repeat_interleave(torch.arange(s["seqs"], device="cuda"), (s["cu"][1:] - s["cu"][:-1]).long())
        outs["pos"] = depth + s["lens"][seq] - (s["cu"][1:] - s["cu"][:-1])[seq]
    if s["lse"]:
        outs["lse"] = lse
    return outs


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "turn":
        pos = _exact_positions(s)
        return {"q": _exact_turn(s, s["q"], s["wq"], pos), "k": _exact_turn(s, s["k"], s["wk"], pos)}
    return _exact_cache(s) if case["kind"] == "append" else _exact_attend(s)
