"""Plain numpy forms of the 8-bit serving operators, written from their
definitions (include/avae.h) for the tests: the quantiser in float32, step by
step as it is defined, everything else in float64."""
import numpy as np

F32 = np.float32


def scale_of(amax):
    """amax times float32's 1 / 127; NaN where amax is not finite."""
    amax = np.asarray(amax, F32)
    return np.where(np.isfinite(amax), amax * (F32(1) / F32(127)), F32(np.nan)).astype(F32)


def quantise(x, scale):
    """rint(x / scale) in float32 arithmetic, 0 where the scale is 0 or NaN."""
    x, scale = np.broadcast_arrays(np.asarray(x, F32), np.asarray(scale, F32))
    ok = scale > 0
    with np.errstate(all="ignore"):
        q = np.rint(x / np.where(ok, scale, F32(1)))
    return np.where(ok, np.clip(q, -127, 127), 0).astype(np.int8)


def rows_q8(x, weight=None, residual=None, eps=1e-6):
    """(q, scale in float64 arithmetic, h) of rows given in float32."""
    h = x.astype(F32) if residual is None else x.astype(F32) + residual.astype(F32)
    with np.errstate(all="ignore"):
        v = h if weight is None else h * weight.astype(F32)
        s = scale_of(np.abs(v).max(1))
        q = quantise(v, s[:, None])
        scale = s.astype(np.float64)
        if weight is not None:
            h64 = h.astype(np.float64)
            scale = scale / np.sqrt((h64 * h64).mean(1) + eps)
    return q, scale, h


def linear_q8(a, sa, w, sw, bias=None, act="none"):
    acc = a.astype(np.int64) @ w.astype(np.int64).T
    y = acc * sa.astype(np.float64)[:, None] * sw.astype(np.float64)
    if bias is not None:
        y = y + bias.astype(np.float64)
    if act == "silu":
        with np.errstate(over="ignore"):
            y = y / (1 + np.exp(-y))
    return y


def kv_write(q8, scales, x, table, cu, lens, n_pages, page):
    """Writes x [total, heads, dim] (float32) into q8 and scales in place."""
    for b, t in enumerate(lens):
        n = cu[b + 1] - cu[b]
        start = t - n
        for col in range(max(start, 0) // page, -(-t // page) if n > 0 else 0):
            p = table[b, col] if col < table.shape[1] else -1
            if p < 0 or p >= n_pages:
                continue
            lo, hi = max(start, col * page, 0), min(t, (col + 1) * page)
            if hi <= lo:
                continue
            rows = x[cu[b] + lo - start:cu[b] + hi - start].astype(F32)
            for h in range(q8.shape[1]):
                with np.errstate(all="ignore"):
                    fresh = scale_of(np.abs(rows[:, h]).max())
                held_rows = lo - col * page
                held = F32(scales[p, h]) if held_rows else F32(0)
                s = F32(np.nan) if np.isnan(fresh) or np.isnan(held) else max(held, fresh)
                if held_rows and s > held:
                    q8[p, h, :held_rows] = quantise(q8[p, h, :held_rows].astype(F32) * held, s)
                scales[p, h] = s
                q8[p, h, held_rows:hi - col * page] = quantise(rows[:, h], s)


def kv_read(q8, scales, table, cu, lens, page):
    """[total, heads, dim] float32 (the product of value and scale)."""
    out = np.zeros((cu[-1], q8.shape[1], q8.shape[3]), F32)
    for b, t in enumerate(lens):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            pos = t - n + i
            col = pos // page
            p = table[b, col] if pos >= 0 and col < table.shape[1] else -1
            if 0 <= p < q8.shape[0]:
                with np.errstate(all="ignore"):
                    out[cu[b] + i] = q8[p, :, pos % page].astype(F32) * scales[p][:, None]
    return out


def attention(q, k8, ks, v8, vs, table, cu, lens, page, scale, causal=True, window=0, first=None):
    """(out, lse, weight, size) in float64: the rows' attention, log sum of
    exponentials, sum_t p_t |v_t| and the largest sum_d |q_d k_d| * |scale|."""
    total, hq, d = q.shape
    hk = k8.shape[1]
    out = np.zeros((total, hq, d))
    weight = np.zeros((total, hq, d))
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
                see = there & (key >= (first[b] if first is not None else 0))
                if causal:
                    see &= key <= pos
                if window:
                    see &= key > pos - window
                if not see.any():
                    continue
                for r in range(h * (hq // hk), (h + 1) * (hq // hk)):
                    x = q[cu[b] + i, r].astype(np.float64)
                    s = scale * (k[see] @ x)
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    out[cu[b] + i, r] = (p / l) @ v[see]
                    weight[cu[b] + i, r] = (p / l) @ np.abs(v[see])
                    lse[cu[b] + i, r] = m + np.log(l)
                    size[cu[b] + i, r] = abs(scale) * (np.abs(k[see]) @ np.abs(x)).max()
    return out, lse, weight, size
