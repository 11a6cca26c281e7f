"""The 8-bit serving operators of an autoregressive latent generator, as cases that can be timed and checked.

A generator that writes the decoder's latent frames one after the other (40 frames a second, so 2400 a minute) runs the same few
operators in each of its layers: the norm of the residual stream with an 8-bit output, products of 8-bit activations and weights, the
write of the new tokens' keys and values into an 8-bit paged cache, and attention over that cache.  `run` computes one of them, in
elementary torch operations where `own` is false and through the library's entry points where it is true.

Kinds of cases and what they return:
  norm    residual sum, and the values that the 8-bit rows stand for
  linear  the product, scaled, with bias and activation
  cache   keys and values of every page that the new tokens went into, read back after the write
  attend  the attention's output rows
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one generated frame of one stream: a single row at the decoder's conv_pre width
        dict(name="norm-step", kind="norm", rows=1, width=1536, dtype="bf16", residual=True, norm=True),
        # a prompt of 150 seconds of frames for one stream, the residual added and kept
        dict(name="norm-prompt", kind="norm", rows=6000, width=1536, dtype="bf16", residual=True, norm=True),
        # the hidden rows of an odd number of tokens, quantised without a norm before the second product of a block
        dict(name="quant-odd", kind="norm", rows=2049, width=5461, dtype="f32", residual=False, norm=False),
        # one frame through the packed query, key and value weights
        dict(name="linear-step", kind="linear", rows=1, n=4608, k=1536, dtype="bf16", bias=False, act="none"),
        # 37 streams' frames through a block's second product, float output
        dict(name="linear-batch", kind="linear", rows=37, n=1536, k=6144, dtype="f32", bias=True, act="none"),
        # a prompt through a block's first product with its activation
        dict(name="linear-prompt", kind="linear", rows=6000, n=6144, k=1536, dtype="bf16", bias=True, act="silu"),
        # 64 streams append one frame each, most of them into pages that hold frames already
        dict(name="cache-append", kind="cache", seqs=64, new_lo=1, new_hi=1, past_hi=2400, kv_heads=4, dim=128, page=64, dtype="bf16"),
        # three ragged prompts are written, one of them after a past
        dict(name="cache-prompt", kind="cache", seqs=3, new_lo=2000, new_hi=6000, past_hi=700, kv_heads=16, dim=64, page=32, dtype="f32"),
        # one stream's next frame after a minute
        dict(name="attend-step", kind="attend", seqs=1, q_lo=1, q_hi=1, past_lo=2399, past_hi=2399, heads=12, kv_heads=4, dim=128, page=64, window=0, dtype="bf16"),
        # 64 streams of up to ten minutes, a frame each
        dict(name="attend-batch", kind="attend", seqs=64, q_lo=1, q_hi=1, past_lo=200, past_hi=24000, heads=12, kv_heads=4, dim=128, page=64, window=0, dtype="bf16"),
        # two prompts of about 100 seconds after as much past
        dict(name="attend-prompt", kind="attend", seqs=2, q_lo=3500, q_hi=4000, past_lo=0, past_hi=4000, heads=12, kv_heads=12, dim=128, page=64, window=0, dtype="bf16"),
        # short drafts checked at once in float32, with a sliding window over small pages
        dict(name="attend-window", kind="attend", seqs=5, q_lo=3, q_hi=17, past_lo=100, past_hi=1900, heads=16, kv_heads=2, dim=64, page=16, window=513, dtype="f32"),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v + 1 if v == 3072 else v


def _drawn(rng):
    kind = rng.choice(["norm", "linear", "cache", "attend"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if kind == "norm":
        norm = rng.random() < 0.7
        return dict(kind=kind, rows=_log(rng, 1, 8192), width=_log(rng, 48, 8200), dtype=dtype, residual=norm and rng.random() < 0.7, norm=norm)
    if kind == "linear":
        k, n = _log(rng, 32, 8192), _log(rng, 48, 8192)
        if rng.random() < 0.7:  # most widths are multiples of 64, some are not
            k, n = max(64, k // 64 * 64), max(64, n // 64 * 64)
        k, n = (v + 64 if v == 3072 else v for v in (k, n))
        return dict(kind=kind, rows=_log(rng, 1, 6000), n=n, k=k, dtype=dtype, bias=rng.random() < 0.5, act=rng.choice(["none", "silu"]))
    kv_heads, dim, page = rng.choice([1, 2, 4, 8, 12]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if kind == "cache":
        seqs = _log(rng, 1, 96)
        hi = 1 if rng.random() < 0.4 else _log(rng, 2, 6000)
        return dict(kind=kind, seqs=seqs, new_lo=max(1, hi // 3), new_hi=hi, past_hi=_log(rng, 1, 5000), kv_heads=kv_heads, dim=dim, page=page, dtype=dtype)
    group = rng.choice([1, 2, 3, 4, 8])
    hi = 1 if rng.random() < 0.5 else _log(rng, 2, 4000)
    past = _log(rng, 16, 24000)
    return dict(kind=kind, seqs=_log(rng, 1, 64), q_lo=max(1, hi // 2), q_hi=hi, past_lo=past // rng.choice([1, 2, 20]), past_hi=past, heads=kv_heads * group,
                kv_heads=kv_heads, dim=dim, page=page, window=rng.choice([0, 0, 0, _log(rng, 32, 2000)]), dtype=dtype)


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
        if w["bytes"] <= b and w["flops"] <= f and _padded(c) <= 3e9:
            return c


def _padded(case):
    """Values of the largest array that the plain form of an attention makes."""
    if case["kind"] != "attend":
        return 0.0
    new, total = _lengths(case)
    return float(case["seqs"]) * max(total) * max(case["heads"] * max(new), case["kv_heads"] * case["dim"])


def _lengths(case):
    """New tokens and length afterwards of each sequence: by the case alone, so that what it asks for is known."""
    r = random.Random("%d %d %d" % (case["seqs"], case["past_hi"], case["page"]))
    lo, hi = (case["new_lo"], case["new_hi"]) if case["kind"] == "cache" else (case["q_lo"], case["q_hi"])
    new = [r.randint(lo, hi) for _ in range(case["seqs"])]
    past = [r.randint(case.get("past_lo", 0), case["past_hi"]) for _ in range(case["seqs"])]
    return new, [a + b for a, b in zip(new, past)]


def work(case):
    es = SIZE[case["dtype"]]
    if case["kind"] == "norm":
        m = case["rows"] * case["width"]
        return {"bytes": m * es * (4 if case["residual"] else 2) + 4 * case["width"] * case["norm"], "flops": 0}
    if case["kind"] == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        return {"bytes": m * k + n * k + m * n * es + 4 * (m + n + n * case["bias"]), "flops": 2 * m * n * k}
    new, total = _lengths(case)
    row = case["kv_heads"] * case["dim"]
    if case["kind"] == "cache":
        back = sum(t - (t - n) // case["page"] * case["page"] for n, t in zip(new, total))
        # new rows in, their 8-bit values out, and the touched pages' rows out once more as the values they stand for
        return {"bytes": 2 * row * (sum(new) * (es + 1) + back * (1 + es)), "flops": 0}
    pairs = keys = 0
    w = case["window"]
    for n, t in zip(new, total):
        first = t - n
        pairs += sum(min(w, p + 1) for p in range(first, t)) if w else (first + 1 + t) * n // 2
        keys += min(t, n + w - 1) if w else t
    return {"bytes": 2 * row * keys + 2 * sum(new) * case["heads"] * case["dim"] * es, "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    if case["kind"] == "norm":
        m, c = case["rows"], case["width"]
        # a residual stream: a few channels are much larger than the others
        spread = torch.exp(0.7 * _normal(g, c))
        s["x"] = (_normal(g, m, c) * spread).to(dt)
        s["res"] = (_normal(g, m, c) * 2 * spread).to(dt) if case["residual"] else None
        s["w"] = 1 + 0.2 * _normal(g, c) if case["norm"] else None
        return s
    if case["kind"] == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        s["a"] = (_normal(g, m, k) * 34).round().clamp(-127, 127).to(torch.int8)
        s["b"] = (_normal(g, n, k) * 34).round().clamp(-127, 127).to(torch.int8)
        s["sa"] = torch.exp(0.3 * _normal(g, m)) * 0.03
        s["sb"] = torch.exp(0.3 * _normal(g, n)) * (1 / (34 * math.sqrt(k)))
        s["bias"] = 0.1 * _normal(g, n) if case["bias"] else None
        return s
    new, total = _lengths(case)
    b, h, d, p = case["seqs"], case["kv_heads"], case["dim"], case["page"]
    pages = [-(-t // p) for t in total]
    count = sum(pages) + 3  # a few pages belong to nobody
    order = torch.randperm(count, generator=g, device="cuda").to(torch.int32)[: sum(pages)].cpu()
    table = torch.full((b, max(pages)), -1, dtype=torch.int32)
    at = 0
    for i, c in enumerate(pages):
        table[i, :c] = order[at : at + c]
        at += c
    s["table"] = table.cuda()
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    s["total"], s["max_new"], s["max_len"] = cu[-1], max(new), max(total)
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
    if case["kind"] == "attend":
        s["q"] = _normal(g, s["total"], case["heads"], d).to(dt)
        return s
    s["k"] = (_normal(g, s["total"], h, d) * wide[:, 0]).to(dt)
    s["v"] = _normal(g, s["total"], h, d).to(dt)
    # every token of the pages that the new ones go into is read back
    back = [t - (t - n) // p * p for n, t in zip(new, total)]
    cu = [0]
    for n in back:
        cu.append(cu[-1] + n)
    s["back"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["back_total"], s["max_back"] = cu[-1], max(back)
    return s


# ------------------------------------------------------------------ plain forms

def _quantise(x, amax):
    """Rows of 8-bit values with one float32 scale each: the largest magnitude stands at 127."""
    scale = amax / 127
    q = torch.where(scale > 0, (x / scale).round(), 0.0).clamp(-127, 127)
    return q, scale


def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    if s["w"] is None:
        q, scale = _quantise(h, h.abs().amax(1, keepdim=True))
    else:
        rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        v = h * s["w"]
        q, scale = _quantise(v, v.abs().amax(1, keepdim=True))
        scale = scale * rstd
    out = {"y": (q * scale).to(s["x"].dtype)}
    if s["res"] is not None:
        out["sum"] = h.to(s["x"].dtype)
    return out


def _plain_linear(s):
    y = s["a"].float() @ s["b"].float().t()
    y = y * s["sa"][:, None] * s["sb"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    return y.to(DTYPES[s["dtype"]])


def _places(s, cu, total):
    """Sequence and position of each packed token: a sequence's tokens are its last ones."""
    tok = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu[1:].long(), tok, right=True)
    pos = s["lens"].long()[seq] - cu.long()[seq + 1] + tok
    return seq, pos


def _plain_write(s, x, q8, scales):
    p = s["page"]
    x = x.float()
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
    return (q8[page, :, pos % s["page"]].float() * scales[page][:, :, None]).to(DTYPES[s["dtype"]])


def _plain_cache(s):
    _plain_write(s, s["k"], s["k8"], s["ks"])
    _plain_write(s, s["v"], s["v8"], s["vs"])
    return {"k": _plain_read(s, s["k8"], s["ks"]), "v": _plain_read(s, s["v8"], s["vs"])}


def _plain_attend(s):
    b, h, d, p = s["seqs"], s["kv_heads"], s["dim"], s["page"]
    group, n = s["heads"] // h, s["max_new"]
    table = s["table"].long().clamp(min=0)

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
    at = torch.full((b, n), -1, device="cuda")
    at[seq, row] = pos
    key = torch.arange(keys.shape[2], device="cuda")
    seen = key <= at[:, :, None]
    if s["window"]:
        seen &= key > at[:, :, None] - s["window"]
    seen = seen[:, None, :, None].expand(-1, -1, -1, group, -1).reshape(b, 1, n * group, -1)
    scores = scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(3, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    scores = torch.exp_(scores.sub_(top))
    total = scores.sum(3, keepdim=True)
    out = (scores @ values) / torch.where(total > 0, total, 1.0)
    out = out.view(b, h, n, group, d).transpose(1, 2)[seq, row]
    return out.reshape(-1, s["heads"], d).to(DTYPES[s["dtype"]])


def _own(s):
    from bigvgan_waveform_decoder_amd import avae

    if s["kind"] == "norm":
        if s["w"] is None:
            q, scale = avae.quant_q8(s["x"])
            return {"y": avae.dequant_q8(q, scale, dtype=s["x"].dtype)}
        q, scale, h = avae.rms_norm_q8(s["x"], s["w"], eps=EPS, residual=s["res"])
        out = {"y": avae.dequant_q8(q, scale, dtype=s["x"].dtype)}
        if h is not None:
            out["sum"] = h
        return out
    dt = DTYPES[s["dtype"]]
    if s["kind"] == "linear":
        return avae.linear_q8(s["a"], s["sa"], s["b"], s["sb"], bias=s["bias"], act=s["act"], dtype=dt)
    cache = avae.KvCacheQ8(s["k8"], s["v8"], s["ks"], s["vs"])
    if s["kind"] == "cache":
        avae.kv_write_q8(cache, s["k"], s["v"], s["table"], s["cu"], s["lens"], max_new=s["max_new"])
        k, v = avae.kv_read_q8(cache, s["table"], s["back"], s["lens"], total=s["back_total"], max_rows=s["max_back"], dtype=dt)
        return {"k": k, "v": v}
    return avae.attn_q8(s["q"], cache, s["table"], s["cu"], s["lens"], max_q=s["max_new"], max_len=s["max_len"], window=s["window"])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "linear": _plain_linear, "cache": _plain_cache, "attend": _plain_attend}[state["kind"]](state)


# ------------------------------------------------------------------ 64 bits

def _exact_rows(x, scale):
    """x in 8 bits at a scale that is stored in 32."""
    scale = scale.float().double()
    return torch.round(x / scale).clamp(-127, 127), scale


def _exact_cache(s):
    p, outs = s["page"], {}
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    for name in ("k", "v"):
        x, got = s[name].double(), []
        for i, t in enumerate(lens):
            n = cu[i + 1] - cu[i]
            for j in range((t - n) // p, -(-t // p)):
                lo, hi = max(t - n, j * p), min(t, (j + 1) * p)
                rows = x[cu[i] + lo - (t - n) : cu[i] + hi - (t - n)].transpose(0, 1)
                scale = (rows.abs().amax((1, 2)) / 127).float()
                held, was = s[name + "8"][table[i][j], :, : lo - j * p].double(), s[name + "s"][table[i][j]]
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
    for i, t in enumerate(lens):
        n = cu[i + 1] - cu[i]
        pages = s["table"][i, : -(-t // p)].long()
        at = torch.arange(t - n, t, device="cuda")[:, None]
        key = torch.arange(t, device="cuda")
        hidden = key > at
        if s["window"]:
            hidden = hidden | (at - key >= s["window"])
        for h in range(s["kv_heads"]):
            k = (s["k8"][pages, h].double() * s["ks"][pages, h].double()[:, None, None]).reshape(-1, d)[:t]
            v = (s["v8"][pages, h].double() * s["vs"][pages, h].double()[:, None, None]).reshape(-1, d)[:t]
            for r in range(h * group, (h + 1) * group):
                x = torch.mm(s["q"][cu[i] : cu[i + 1], r].double(), k.t()) * d**-0.5
                x[hidden] = -math.inf
                out[cu[i] : cu[i + 1], r] = torch.mm(torch.softmax(x, 1), v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "norm":
        h = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
        v = h if s["w"] is None else h * s["w"].double()
        q, scale = _exact_rows(v, v.abs().amax(1, keepdim=True) / 127)
        if s["w"] is not None:
            scale = scale / torch.sqrt((h * h).sum(1, keepdim=True) / case["width"] + EPS)
        return {"y": q * scale} if s["res"] is None else {"y": q * scale, "sum": h}
    if case["kind"] == "linear":
        y = torch.mm(s["a"].double(), s["b"].double().t())  # whole numbers below 2^53: exact
        y = y * s["sb"].double() * s["sa"].double()[:, None]
        if s["bias"] is not None:
            y = y + s["bias"].double()
        return y * torch.sigmoid(y) if case["act"] == "silu" else y
    return _exact_cache(s) if case["kind"] == "cache" else _exact_attend(s)
