"""Plain fp64 sliding-window attention with sinks, its gradient, rotary
positions and the rolling cache, one head at a time (numpy; shares no code with
the CUDA side), with bounds on what a kernel's roundings may add.

A rounding to a type is off by at most u = eps / 2 of the value (bf16 2^-8, fp32
2^-24).  With bf16 storage the kernels round P (forward) resp. P and dS
(backward) to bf16 for the tensor cores, and every result once at its end; the
rest is fp32: dot products of d or of up to n terms, each term off by at most
(number of additions) * 2^-24, and the exponential, whose argument x carries an
error of up to e_x = 2^-24 (d + 8) A with A = scale sum|q||k| + |LSE| (the dot
product, the scaling, the subtraction, the row statistics), so that P is off by
a factor of 1 + 2 e_x + 2^-20 (the last for the exponential function itself and
the row sum's division).  First-order terms are added up in absolute values."""
from __future__ import annotations

import math

import numpy as np

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U32 = 2.0 ** -24


def visible(q_len, kv_len, window, sinks):
    p = kv_len - q_len + np.arange(q_len)[:, None]
    j = np.arange(kv_len)[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def _scores(q, k, scale, see):
    s = q @ k.T * scale
    return np.where(see, s, -np.inf)


def attention(q, k, v, scale, window, sinks, u=0.0):
    """One head: O, LSE and the bounds of their errors (u: the storage type's)."""
    see = visible(len(q), len(k), window, sinks)
    s = _scores(q, k, scale, see)
    lse = np.full(len(q), -np.inf)
    some = see.any(-1)
    if some.any():
        m = s[some].max(-1)
        lse[some] = m + np.log(np.exp(s[some] - m[:, None]).sum(-1))
    p = np.where(see, np.exp(s - np.where(some, lse, 0.0)[:, None]), 0.0)
    o = p @ v
    n = len(k)
    a = abs(scale) * (np.abs(q) @ np.abs(k).T)
    ex = _ex(q.shape[1], a, lse, see)
    up = u if u > U32 else U32                          # P's own rounding
    bo = u * np.abs(o) + (p * (up + 2 * ex + 2.0 ** -20 + n * U32)) @ np.abs(v)
    bl = (p * (2 * ex)).sum(-1) + 2.0 ** -20 + n * U32 + U32 * np.abs(np.where(some, lse, 0.0))
    return o, lse, bo, bl


def _ex(d, a, lse, see):
    return np.where(see, U32 * (d + 8) * (np.abs(a) + np.abs(np.where(np.isinf(lse), 0.0, lse))[:, None]), 0.0)


def gradient(q, k, v, o, lse, do, scale, window, sinks, u=0.0):
    """One query head against one key head: dQ, dK, dV and the bounds of their errors
    (without the final rounding of dK and dV, which follows the sum over heads)."""
    see = visible(len(q), len(k), window, sinks)
    s = _scores(q, k, scale, see)
    p = np.where(see, np.exp(s - np.where(np.isinf(lse), 0.0, lse)[:, None]), 0.0)
    dp = do @ v.T
    D = (do * o).sum(-1, keepdims=True)
    ds = p * (dp - D)
    dq, dk, dv = scale * ds @ k, scale * ds.T @ q, p.T @ do
    d, n = q.shape[1], max(len(k), len(q))
    a = abs(scale) * (np.abs(q) @ np.abs(k).T)
    rel = 2 * _ex(d, a, lse, see) + 2.0 ** -20 + n * U32
    up = u if u > U32 else U32
    mag = np.abs(do) @ np.abs(v).T + np.abs(do * o).sum(-1, keepdims=True)
    eds = np.abs(ds) * (2 * up + rel) + p * (mag * U32 * (d + 8))
    bq = u * np.abs(dq) + abs(scale) * eds @ np.abs(k)
    bk = abs(scale) * eds.T @ np.abs(q)
    bv = (p * (up + rel)).T @ np.abs(do)
    return dq, dk, dv, bq, bk, bv


def batch_forward(q, k, v, scale, window, sinks, q_lens, kv_lens, u):
    """[B, Hq, Nq, d] arrays: O, LSE and bounds; padding rows 0 and -inf."""
    B, Hq, Nq, d = q.shape
    G = Hq // k.shape[1]
    o, bo = np.zeros(q.shape), np.zeros(q.shape)
    lse, bl = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    for b in range(B):
        ql, kl = q_lens[b], kv_lens[b]
        for h in range(Hq):
            r = attention(q[b, h, :ql], k[b, h // G, :kl], v[b, h // G, :kl], scale, window, sinks, u)
            o[b, h, :ql], lse[b, h, :ql], bo[b, h, :ql], bl[b, h, :ql] = r
    return o, lse, bo, bl


def batch_gradient(q, k, v, o, lse, do, scale, window, sinks, q_lens, kv_lens, u):
    B, Hq = q.shape[:2]
    G = Hq // k.shape[1]
    dq, bq = np.zeros(q.shape), np.zeros(q.shape)
    dk, dv, bk, bv = (np.zeros(k.shape) for _ in range(4))
    for b in range(B):
        ql, kl = q_lens[b], kv_lens[b]
        for h in range(Hq):
            g = h // G
            r = gradient(q[b, h, :ql], k[b, g, :kl], v[b, g, :kl], o[b, h, :ql], lse[b, h, :ql], do[b, h, :ql], scale,
                         window, sinks, u)
            dq[b, h, :ql], bq[b, h, :ql] = r[0], r[3]
            for to, x in ((dk, r[1]), (dv, r[2]), (bk, r[4]), (bv, r[5])):
                to[b, g, :kl] += x
    bk += np.abs(dk) * (u + G * U32)
    bv += np.abs(dv) * (u + G * U32)
    return dq, dk, dv, bq, bk, bv


def rotation(x, pos, sections, theta, per_axis, interleaved, inverse):
    """x [B, H, N, d], pos [axes, B, N] integers: the rotated x and the error bound's
    factor per element (|x1| + |x2| of its pair)."""
    n = sum(sections)
    y, mag = x.astype(np.float64).copy(), np.abs(x).astype(np.float64)
    i = 0
    for a, s in enumerate(sections):
        for k in range(s):
            f = theta ** -(k / s if per_axis else i / n)
            # modulo a turn in integers: the position times the turn fraction in 2^-70
            frac = int(f / (2 * math.pi) * 2.0 ** 70)
            turn = np.vectorize(lambda p: (int(p) * frac % 2 ** 70) / 2.0 ** 70, otypes=[float])(pos[a])
            ang = (2 * math.pi * turn)[:, None]                    # [B, 1, N]
            c, sn = np.cos(ang), np.sin(ang) * (-1 if inverse else 1)
            f1, f2 = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            x1, x2 = x[..., f1].astype(np.float64), x[..., f2].astype(np.float64)
            y[..., f1], y[..., f2] = x1 * c - x2 * sn, x2 * c + x1 * sn
            mag[..., f1] = mag[..., f2] = np.abs(x1) + np.abs(x2)
            i += 1
    return y, mag


def slot(p, capacity, sinks):
    return p if p < sinks else sinks + (p - sinks) % (capacity - sinks)
