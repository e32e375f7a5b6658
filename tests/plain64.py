"""Plain 64-bit forms of the cache operators and the residual norms, in numpy
loops over rows and requests, with the bounds that fp32 results are held to.

HALF is the largest relative error of one rounding, by type."""
import numpy as np

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def assign(lengths, delta, table, free, count, page, rows):
    """kv_assign on lists; returns None where the step does not fit."""
    n = len(lengths)
    table, free = [list(r) for r in table], list(free)
    new = [max(0, int(a) + int(d)) for a, d in zip(lengths, delta)]
    width = len(table[0])
    pages = [-(-int(x) // page) for x in lengths]
    need = [-(-x // page) for x in new]
    if min(lengths) < 0 or max(pages) > width or max(need) > width or max(new) >= 2 ** 31:
        return None
    back = [table[r][j] for r in range(n) for j in range(need[r], pages[r])]
    taken = sum(max(0, b - a) for a, b in zip(pages, need))
    total = sum(max(0, b - int(a)) for a, b in zip(lengths, new))
    if count < 0 or count + len(back) > len(free) or taken > count + len(back) or total > rows:
        return None
    free[count:count + len(back)] = back
    top = count + len(back)
    for r in range(n):
        for j in range(pages[r], need[r]):
            top -= 1
            table[r][j] = free[top]
    slots, positions, requests, start = [-1] * rows, [0] * rows, [-1] * rows, [0]
    t = 0
    for r in range(n):
        for p in range(int(lengths[r]), new[r]):
            slots[t] = table[r][p // page] * page + p % page
            positions[t], requests[t] = p, r
            t += 1
        start.append(t)
    return dict(lengths=new, free_count=[top], block_table=table, free_pages=free, slots=slots,
                positions=positions, requests=requests, row_start=start)


def rotate(x, positions, inv_freq, interleaved):
    """x [rows, heads, d] in 64 bits, and a bound on what fp32 makes of it: the
    reduced angle is off by half a step below pi (2^-23), sine and cosine by
    two steps below 1 (2^-23), and a product, a product and a sum by one
    rounding each (2^-24): together 7 * 2^-24 of |a| + |b|."""
    out, tol = x.astype(np.float64).copy(), np.zeros(x.shape)
    half = len(inv_freq)
    if not half:
        return out, tol
    a_at, b_at = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else \
        (np.arange(half), np.arange(half) + half)
    ang = np.outer(np.asarray(positions, np.float64), inv_freq)[:, None, :]
    a, b = x[..., a_at].astype(np.float64), x[..., b_at].astype(np.float64)
    out[..., a_at] = a * np.cos(ang) - b * np.sin(ang)
    out[..., b_at] = b * np.cos(ang) + a * np.sin(ang)
    tol[..., a_at] = tol[..., b_at] = 7 * 2.0 ** -24 * (np.abs(a) + np.abs(b))
    return out, tol


def attention(q, k, v, scale, heads, v_scale=None):
    """One request: q [heads, d], k and v [n, kv_heads, d] in 64 bits.  Returns
    out, lse and their bounds.

    A score is a sum of d products whose q is carried in 21 bits or more
    (2^-22 of each term) in fp32 (d + 2 roundings of the partial sums, each at
    most 2^-24 of the terms' magnitudes), and its distance to the maximum is
    rounded at its own size: e = scale * sum|q k| * (2^-22 + (d + 2) 2^-24) +
    2^-23 max|s|.  A weight is then off by 2 e and the exponential's own error
    (2^-21, the rescalings with it), and carried in 21 bits (2^-22); the sums
    over n keys add n roundings at most (2^-24 each).  All of that relative to
    sum p |v|; the division adds one rounding, the sum of weights the same
    errors again.

    fp16 operands end at 2^-24.  The largest weight is carried at 2^12 or
    more, so that any weight is off by half of fp16's last step at most: by
    2^-25 / 2^12 = 2^-37 of the largest, for each key times its value.  Over
    codes it is weight times v_scale [n, kv_heads] that is carried, to 2^-37
    of its largest, times the code."""
    n = k.shape[0]
    group = heads // k.shape[1] if k.ndim == 3 else 1
    d = q.shape[1]
    out, lse = np.zeros((heads, d)), np.full(heads, -np.inf)
    out_tol, lse_tol = np.zeros((heads, d)), np.zeros(heads)
    for h in range(heads if n else 0):
        kk, vv = k[:, h // group], v[:, h // group]
        s = scale * (kk @ q[h])
        m = s.max()
        p = np.exp(s - m)
        out[h] = (p / p.sum()) @ vv
        lse[h] = m + np.log(p.sum())
        e = abs(scale) * (np.abs(kk) @ np.abs(q[h])).max() * (2.0 ** -22 + (d + 2) * 2.0 ** -24) \
            + 2.0 ** -23 * np.abs(s).max()
        rel = 2 * e + 2.0 ** -21 + 2.0 ** -22 + n * 2.0 ** -24
        vs = np.ones(n) if v_scale is None else np.where(v_scale[:, h // group] > 0, v_scale[:, h // group], 1.0)
        tiny = 2.0 ** -37 * (p * vs).max() * (np.abs(vv) / vs[:, None]).sum(axis=0) / p.sum()
        out_tol[h] = 2 * rel * ((p / p.sum()) @ np.abs(vv)) + tiny + 1e-38
        lse_tol[h] = rel + 2.0 ** -23 * (abs(lse[h]) + abs(m))
    return out, lse, out_tol, lse_tol


def norm(u, du, kind, w, b, eps):
    """Norm of rows u [m, k] known to within du; its value and bound.  A sum
    of k values in fp32 passes at most SUM roundings: a thread's own (128
    values at most), ten in the butterfly and the warps' values in order."""
    SUM = 128 + 10 + 32
    r24 = 2.0 ** -24
    if kind is None:
        return u, du
    k = u.shape[1]
    if kind == "layer":
        mean = u.mean(axis=1, keepdims=True)
        dm = np.abs(u).mean(axis=1, keepdims=True) * (SUM + 2) * r24 + du.mean(axis=1, keepdims=True)
        u = u - mean
        du = du + dm + np.abs(u) * r24
    ms = (u * u).mean(axis=1, keepdims=True) + eps
    # the mean square: its own roundings, and what du changes in it
    dms = ms * (SUM + 4) * r24 + 2 * (np.abs(u) * du).mean(axis=1, keepdims=True) + \
        (du * du).mean(axis=1, keepdims=True)
    r = 1 / np.sqrt(ms)
    dr = r * (dms / ms + 3 * r24)   # half of it by the root; a factor two left for large dms / ms
    w = np.ones(k) if w is None else w
    n = u * r * w
    dn = np.abs(w) * (du * (r + dr) + np.abs(u) * dr) + 3 * r24 * np.abs(n)
    if b is not None:
        n = n + b
        dn = dn + r24 * np.abs(n)
    return n, dn


def residual_norm(x, y, post, pw, pb, gate, alpha, pre, w, b, eps):
    """h, n and their bounds."""
    r24 = 2.0 ** -24
    h, dh = x, np.zeros(x.shape)
    if y is not None:
        t, dt = norm(y, np.zeros(y.shape), post, pw, pb, eps)
        if gate is not None:
            t, dt = t * gate, np.abs(gate) * dt + r24 * np.abs(t * gate)
        h = x + alpha * t
        dh = abs(alpha) * dt + r24 * (np.abs(h) + np.abs(alpha * t))
    n, dn = norm(h, dh, pre, w, b, eps)
    return h, n, dh, dn
