"""Plain numpy forms in float64 of the operators that turn heads by their
position and of the attention with rules, written from their definitions
(include/avae.h) for the tests."""
import math

import numpy as np


def turn(x, pos, freq, interleaved=False, amp=1.0, weight=None, eps=1e-6):
    """x [tokens, heads, dim] normed (with a weight) and turned, and what the
    magnitudes |a| + |b| of each value's pair are (times amp), for tolerances."""
    x = x.astype(np.float64)
    with np.errstate(all="ignore"):
        if weight is not None:
            r = np.sqrt((x * x).mean(2, keepdims=True) + eps)
            x = np.where(r > 0, x / np.where(r > 0, r, 1), 0) * weight.astype(np.float64)
        out, size = x.copy(), np.abs(x)
        half = len(freq)
        angle = np.asarray(pos, np.float64)[:, None] * np.asarray(freq, np.float64)
        c, s = (np.cos(angle) * amp)[:, None], (np.sin(angle) * amp)[:, None]
        at = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (
            slice(0, half), slice(half, 2 * half))
        a, b = x[..., at[0]], x[..., at[1]]
        out[..., at[0]], out[..., at[1]] = a * c - b * s, b * c + a * s
        for i in at:
            size[..., i] = abs(amp) * (np.abs(a) + np.abs(b))
    return out, size


def rope_freq(rot, theta, scaling="plain", factor=1.0, context=4096.0, low=1.0, high=32.0):
    half = rot // 2
    out = []
    if scaling == "base":
        theta *= factor ** (rot / (rot - 2))
    first = last = 0.0
    if scaling == "ramp":
        index = [half * math.log(context / (2 * math.pi * t)) / math.log(theta) for t in (high, low)]
        first, last = max(math.floor(index[0]), 0), min(math.ceil(index[1]), rot - 1)
    for i in range(half):
        f = theta ** (-2 * i / rot)
        w = {"linear": 0.0, "bands": (context * f / (2 * math.pi) - low) / (high - low),
             "ramp": 1 - (i - first) / max(last - first, 1e-3)}.get(scaling, 1.0)
        w = min(max(w, 0.0), 1.0)
        out.append(f if scaling == "base" else f * w + f / factor * (1 - w))
    return np.array(out), 0.1 * math.log(factor) + 1 if scaling == "ramp" else 1.0


def lineage(parents, cu):
    """[list of the drafts that draft i sees, itself the last] by their
    parents; a parent that does not come before its child is none."""
    out = []
    for b in range(len(cu) - 1):
        for i in range(cu[b + 1] - cu[b]):
            p = parents[cu[b] + i]
            out.append((out[cu[b] + p] if 0 <= p < i else []) + [i])
    return out


def tree_words(lines, words):
    """Masks [tokens, words] int32 of lists of drafts."""
    out = np.zeros((len(lines), words), np.uint32)
    for i, line in enumerate(lines):
        for j in line:
            out[i, j // 32] |= np.uint32(1 << (j % 32))
    return out.view(np.int32)


def attention(q, k8, ks, v8, vs, table, cu, lens, page, scale, causal=True, window=0, first=None,
              cap=0.0, slopes=None, prefix=None, lines=None):
    """(out, lse, weight, size, bent): as q8_reference.attention, and
    sum_t p_t (|v_t| + sum_u p_u |v_u|) |slope (p - t)|."""
    total, hq, d = q.shape
    hk = k8.shape[1]
    out, weight, bent = np.zeros((total, hq, d)), np.zeros((total, hq, d)), np.zeros((total, hq, d))
    lse = np.full((total, hq), -np.inf)
    size = np.zeros((total, hq))
    for b, t in enumerate(lens):
        n = cu[b + 1] - cu[b]
        if n <= 0 or t <= 0:
            continue
        pages = [table[b, c] if c < table.shape[1] else -1 for c in range(-(-t // page))]
        there = np.repeat([0 <= p < k8.shape[0] for p in pages], page)[:t]
        at = np.array([p if 0 <= p < k8.shape[0] else 0 for p in pages])
        key = np.arange(t)
        for h in range(hk):
            with np.errstate(invalid="ignore"):
                k = (k8[at, h].astype(np.float64) * ks[at, h].astype(np.float64)[:, None, None]
                     ).reshape(-1, d)[:t]
                v = (v8[at, h].astype(np.float64) * vs[at, h].astype(np.float64)[:, None, None]
                     ).reshape(-1, d)[:t]
            for i in range(n):
                pos = t - n + i
                if pos < 0:
                    continue
                if lines is not None:
                    see = key < t - n
                    mine = [t - n + j for j in lines[cu[b] + i] if j < n and t - n + j >= 0]
                    see[mine] = True
                else:
                    see = key <= pos if causal else key >= 0
                    if window:
                        see &= key > pos - window
                    if prefix is not None:
                        see |= key < prefix[b]
                see &= there & (key >= (first[b] if first is not None else 0))
                if not see.any():
                    continue
                for r in range(h * (hq // hk), (h + 1) * (hq // hk)):
                    x = q[cu[b] + i, r].astype(np.float64)
                    s = scale * (k[see] @ x)
                    if cap:
                        s = cap * np.tanh(s / cap)
                    far = np.zeros(see.sum())
                    if slopes is not None:
                        far = slopes[r].astype(np.float64) * np.abs(pos - key[see])
                        s = s - far
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    p /= l
                    with np.errstate(invalid="ignore"):
                        out[cu[b] + i, r] = p @ v[see]
                        w = p @ np.abs(v[see])
                        weight[cu[b] + i, r] = w
                        bent[cu[b] + i, r] = (p * np.abs(far)) @ (np.abs(v[see]) + w)
                    lse[cu[b] + i, r] = m + np.log(l)
                    size[cu[b] + i, r] = abs(scale) * (np.abs(k[see]) @ np.abs(x)).max()
    return out, lse, weight, size, bent
