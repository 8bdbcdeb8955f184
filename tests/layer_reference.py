"""Plain fp64 forms of the attention layer's operators (rotary positions, cache append, attention
over the paged cache, block norm), for the tests.  Each returns, next to a result, the sum of the
absolute terms it was made of where a tolerance is derived from them."""
import math

import numpy as np
import torch


def frequencies(rot, base, factor, trained_len, low, high):
    w = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    keep = np.zeros_like(w)
    if trained_len:
        keep = np.clip((trained_len * w / (2 * math.pi) - low) / (high - low), 0, 1)
    return w * (keep + (1 - keep) / factor)


def positions(offsets, kv_len=None):
    """Position of every token of a jagged batch."""
    out = []
    for b in range(len(offsets) - 1):
        n = offsets[b + 1] - offsets[b]
        first = kv_len[b] - n if kv_len is not None else 0
        out += [first + i for i in range(n)]
    return np.array(out, dtype=np.int64)


def rotary(x, pos, rot, interleaved=False, base=10000.0, factor=1.0, trained_len=0, low=1.0,
           high=32.0, mscale=1.0, inverse=False):
    """(rotated, |a| + |b| of each element's pair) for x [T, h, dh] fp64."""
    x = np.asarray(x, dtype=np.float64)
    w = frequencies(rot, base, factor, trained_len, low, high)
    t = np.asarray(pos, dtype=np.float64)[:, None] * w * (-1 if inverse else 1)
    c, s = (mscale * f(t)[:, None, :] for f in (np.cos, np.sin))
    y, mag = x.copy(), np.abs(x)
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    mag[..., first] = mag[..., second] = np.abs(mscale) * (np.abs(a) + np.abs(b))
    return y, mag


def chunk(q, offsets, kv_len, table, cache_k, cache_v, scale, window=None):
    """(o, lse, sum p|v|, bound of a logit's terms scale * sum |q||k|) in fp64."""
    q = np.asarray(q, dtype=np.float64)
    T, hq, dh = q.shape
    _, hk, page, _ = cache_k.shape
    o, mag = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((hq, T), -np.inf)
    size = np.zeros((hq, T))
    pos = positions(offsets, kv_len)
    for b in range(len(offsets) - 1):
        for t in range(offsets[b], offsets[b + 1]):
            lo = max(0, pos[t] - window + 1) if window else 0
            seen = np.arange(lo, pos[t] + 1)
            if not len(seen):
                continue
            pages, rows = table[b][seen // page], seen % page
            for j in range(hq):
                k = cache_k[pages, j // (hq // hk), rows].astype(np.float64)
                v = cache_v[pages, j // (hq // hk), rows].astype(np.float64)
                x = scale * (k @ q[t, j])
                m = x.max()
                p = np.exp(x - m)
                lse[j, t] = m + math.log(p.sum())
                p /= p.sum()
                o[t, j], mag[t, j] = p @ v, p @ np.abs(v)
                size[j, t] = (abs(scale) * (np.abs(k) @ np.abs(q[t, j]))).max()
    return o, lse, mag, size


def act(z, sigmoid):
    return torch.sigmoid(z) if sigmoid else z


def block_norm(x, f=None, gate=None, w_post=None, w_pre=None, sample=None, alpha=1.0, eps=1e-6,
               sigmoid=False):
    """(y, n) in fp64 (torch, differentiable); ``sample``: each row's sample, for a shared gate."""
    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w
    y = x
    if f is not None:
        u = f if w_post is None else norm(f, w_post)
        if gate is not None:
            a = act(gate, sigmoid)
            u = u * (a if sample is None else a[sample])
        y = x + alpha * u
    return y, None if w_pre is None else norm(y, w_pre)


def block_norm_grads(y, f, gate, w_post, w_pre, dy, dn, sample=None, B=0, alpha=1.0, eps=1e-6,
                     sigmoid=False):
    """The gradients by their formulas, each as (value, sum of its absolute terms)."""
    zero = torch.zeros_like(y)
    G, Gm = (zero, zero) if dy is None else (dy, dy.abs())
    out = {}
    if w_pre is not None:
        r = 1 / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        yh, t = y * r, dn * w_pre
        G = G + r * (t - yh * (t * yh).mean(-1, keepdim=True))
        Gm = Gm + r * (t.abs() + yh.abs() * (t * yh).abs().mean(-1, keepdim=True))
        out["dw_pre"] = (dn * yh).sum(0), (dn * yh).abs().sum(0)
    out["dx"] = G, Gm
    if f is None:
        return out
    rf = 1 / torch.sqrt((f * f).mean(-1, keepdim=True) + eps)
    fh = f * rf if w_post is not None else f
    w = torch.ones_like(f[0]) if w_post is None else w_post
    a = torch.ones_like(f) if gate is None else act(gate, sigmoid)
    slope = a * (1 - a) if gate is not None and sigmoid else torch.ones_like(a)
    if sample is not None:
        a, slope = a[sample], slope[sample]
    du, dum = alpha * a * G, abs(alpha) * a.abs() * Gm
    if gate is not None:
        dg, dgm = alpha * slope * G * fh * w, (alpha * slope * fh * w).abs() * Gm
        if sample is not None:
            dg, dgm = (torch.zeros(B, f.shape[1], dtype=f.dtype).index_add_(0, sample, v)
                       for v in (dg, dgm))
        out["dgate"] = dg, dgm
    if w_post is None:
        out["df"] = du, dum
    else:
        t, tm = du * w, dum * w.abs()
        out["df"] = (rf * (t - fh * (t * fh).mean(-1, keepdim=True)),
                     rf * (tm + fh.abs() * (tm * fh.abs()).mean(-1, keepdim=True)))
        out["dw_post"] = (du * fh).sum(0), (dum * fh.abs()).sum(0)
    return out
