"""64-bit oracle of the attention block's operators (test infrastructure only).

Plain numpy from the definitions; every function also returns the magnitude
that a rounding bound is stated against.
"""
from __future__ import annotations

import numpy as np


def norm_rope(x, weight, eps, cos_sin, pos, rot, interleaved):
    """Rows ``x`` [tokens][heads][dim] normed (``weight`` None: not) and
    rotated.  Returns (y, mag): ``mag`` is |y| before the pairs' terms cancel."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    y, mag = x.copy(), np.abs(x)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c = np.asarray(cos_sin, np.float64)[pos, i][:, None]
        s = np.asarray(cos_sin, np.float64)[pos, rot // 2 + i][:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        mag[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, mag


def paged_attn(q, k_cache, v_cache, table, new, kv_len, scale, window=0):
    """q [tokens][heads][dim]; caches [pages][kv_heads][page_size][dim]; table
    [requests][max_pages].  Returns (out, pv, vmax, z): ``pv`` is sum p |v|,
    ``vmax`` the largest |v| that a row sees and ``z`` its largest
    |scale| sum |q||k|."""
    q = np.asarray(q, np.float64)
    out, pv, vmax, mag = np.zeros_like(q), np.zeros_like(q), np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    page, group = k_cache.shape[2], q.shape[1] // k_cache.shape[1]
    t = 0
    for r, (n, kv) in enumerate(zip(new, kv_len)):
        cells = np.arange(kv)
        k = np.asarray(k_cache[table[r][cells // page], :, cells % page], np.float64)     # [kv][kv_heads][dim]
        v = np.asarray(v_cache[table[r][cells // page], :, cells % page], np.float64)
        for i in range(n):
            p = kv - n + i
            lo = max(0, p - window + 1) if window else 0
            if p >= lo:
                for h in range(q.shape[1]):
                    z = k[lo:p + 1, h // group] @ q[t, h] * scale
                    mag[t, h] = (np.abs(k[lo:p + 1, h // group]) @ np.abs(q[t, h])).max() * abs(scale)
                    w = np.exp(z - z.max())
                    w /= w.sum()
                    out[t, h] = w @ v[lo:p + 1, h // group]
                    pv[t, h] = w @ np.abs(v[lo:p + 1, h // group])
                    vmax[t, h] = np.abs(v[lo:p + 1, h // group]).max()
            t += 1
    return out, pv, vmax, mag


def lora_add(x, a, b, base, adapters, scale):
    """x [tokens][cols], a [n][rank][cols], b [n][rows][rank], base
    [tokens][rows] or None.  Returns (y, mag)."""
    x, a, b = (np.asarray(v, np.float64) for v in (x, a, b))
    y = np.zeros((x.shape[0], b.shape[1])) if base is None else np.array(base, np.float64)
    mag = np.abs(y)
    for t, n in enumerate(adapters):
        if n >= 0:
            y[t] += float(scale[n]) * (b[n] @ (a[n] @ x[t]))
            mag[t] += abs(float(scale[n])) * (np.abs(b[n]) @ (np.abs(a[n]) @ np.abs(x[t])))
    return y, mag
