"""fp64 CPU definitions of the cache and window operators (test infrastructure).

Written from the formulas, with numpy; e4m3 and bf16 rounding are written from
the formats' definitions.  Attention results come with the sums that the tests'
error bounds are made of.
"""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0


def e4m3_round(x):
    """Nearest e4m3 value, ties to even, saturated: step 2^(e-3) in [2^e, 2^(e+1)),
    2^-9 below 2^-6.  NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        a = np.minimum(np.abs(x), 1e9)
        e = np.frexp(np.maximum(a, 2.0**-6))[1] - 1
        step = np.ldexp(1.0, e - 3)
        r = np.minimum(np.rint(a / step) * step, E4M3_MAX)
    return np.where(np.isnan(x), np.nan, np.copysign(r, x))


def e4m3_decode(codes):
    """Values of e4m3 codes (s eeee mmm, bias 7, 0x7F and 0xFF NaN)."""
    c = np.asarray(codes, dtype=np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0**-9, np.ldexp(1.0 + m / 8.0, e - 7))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def bf16_round(x):
    """Nearest bf16 value of fp32 values, ties to even."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32)


def token_quantise(x):
    """Rows [..., d] -> (e4m3 values, fp32 scales): scale = max|x|/448 in fp32, 1 for zeros."""
    x = np.asarray(x, dtype=np.float32)
    fin = np.where(np.isfinite(x), np.abs(x), 0).max(-1)
    s = np.where(fin > 0, fin / np.float32(E4M3_MAX), np.float32(1)).astype(np.float32)
    with np.errstate(over="ignore"):
        return e4m3_round((x / s[..., None]).astype(np.float32)), s


def page_power(top):
    """Least power of two p >= 2^-126 with top <= 448 p."""
    p = -126
    while top > E4M3_MAX * 2.0**p:
        p += 1
    return 2.0**p


def paged_write(x, table, start, count, values, scale):
    """x [B,N,Hkv,d]; values [P,Hkv,page,d] (e4m3 values), scale [P,Hkv]: updated in place."""
    P, Hkv, page, d = values.shape
    for b in range(x.shape[0]):
        lo, n = int(start[b]), int(count[b])
        if n < 0 or n > x.shape[1] or lo < 0 or lo + n > table.shape[1] * page:
            continue
        for j in range(lo // page, -(-(lo + n) // page)):
            t0, t1 = max(lo, j * page), min(lo + n, (j + 1) * page)
            pid, a = int(table[b, j]), t0 - j * page
            if t0 >= t1 or not 0 <= pid < P:
                continue
            for h in range(Hkv):
                new = np.asarray(x[b, t0 - lo:t1 - lo, h], dtype=np.float64)
                p = page_power(np.where(np.isfinite(new), np.abs(new), 0).max())
                had = float(scale[pid, h])
                if a > 0 and np.isfinite(had) and had > 0:
                    if p > had:
                        values[pid, h, :a] = e4m3_round(values[pid, h, :a] * (had / p))
                    else:
                        p = had
                values[pid, h, a:a + t1 - t0] = e4m3_round(new / p)
                scale[pid, h] = p


def attend(q, k, v, scale):
    """q [G,d], k/v [n,d] in fp64 -> dict: o [G,d], lse [G], and for the bounds
    av [G,d] = sum p|v|, x [G] = max_s sum_i |q_i k_i| scale, k1 = max_s sum_i |k_i| scale,
    vmax [d]."""
    G, d = q.shape
    if k.shape[0] == 0:
        z = np.zeros((G, d))
        return dict(o=z, lse=np.full(G, -np.inf), av=z, x=np.zeros(G), k1=0.0, vmax=np.zeros(d))
    x = (q @ k.T) * scale
    m = x.max(1, keepdims=True)
    e = np.exp(x - m)
    l = e.sum(1, keepdims=True)
    p = e / l
    return dict(o=p @ v, lse=(m + np.log(l))[:, 0], av=p @ np.abs(v),
                x=(np.abs(q) @ np.abs(k).T).max(1) * scale, k1=np.abs(k).sum(1).max() * scale,
                vmax=np.abs(v).max(0))


def _stack(out, G, d, lead):
    wide = ("o", "av", "vmax")
    return {n: np.concatenate([np.broadcast_to(r[n], (G, d) if n in wide else (G,)) for r in out])
            .reshape(lead + ((d,) if n in wide else ())) for n in out[0]}


def paged_rows(values, scale, table, page, pos):
    """Rows [n, Hkv, d] of one sequence at positions pos; positions on bad pages left out."""
    P = values.shape[0]
    pid = np.asarray(table)[pos // page]
    ok = (pid >= 0) & (pid < P)
    pos, pid = pos[ok], pid[ok]
    return values[pid, :, pos % page] * scale[pid][..., None]


def paged_decode(q, kvals, vvals, kscale, vscale, table, lengths, window, n_sink, sm_scale):
    """q [B,Hq,d].  Returns the dict of attend() stacked to [B,Hq,...]."""
    B, Hq, d = q.shape
    P, Hkv, page, _ = kvals.shape
    G = Hq // Hkv
    out = []
    for b in range(B):
        T = int(lengths[b])
        if not 0 <= T <= table.shape[1] * page:
            T = 0
        pos = np.arange(T)
        pos = pos[(pos >= T - window) | (pos < n_sink)]
        k, v = (paged_rows(z, s, table[b], page, pos) for z, s in ((kvals, kscale), (vvals, vscale)))
        top = paged_rows(np.full_like(vvals, 448.0), vscale, table[b], page, pos)
        for h in range(Hkv):
            r = attend(q[b, h * G:(h + 1) * G], k[:, h], v[:, h], sm_scale)
            r["vmax"] = np.full(d, top[:, h].max() if len(top) else 0.0)  # largest value a code can stand for
            out.append(r)
    return _stack(out, G, d, (B, Hq))


def window_attn(q, k, v, window, n_sink, sm_scale, rows=None):
    """q [B,Lq,Hq,d], k/v [B,Lk,Hkv,d]; rows: the queries to compute (all).
    Returns the dict of attend() stacked to [B,R,Hq,...]."""
    B, Lq, Hq, d = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    rows = range(Lq) if rows is None else rows
    out = []
    for b in range(B):
        for i in rows:
            t = Lk - Lq + i
            s = np.arange(t + 1)
            s = s[(s > t - window) | (s < n_sink)]
            for h in range(Hkv):
                out.append(attend(q[b, i, h * G:(h + 1) * G], k[b, s, h], v[b, s, h], sm_scale))
    return _stack(out, G, d, (B, len(list(rows)), Hq))
