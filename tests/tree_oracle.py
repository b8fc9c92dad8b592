"""Plain fp64 counterparts of the 8-bit cache and of the attention of drafted tokens
(numpy, torch on the CPU for the e4m3 format alone), with bounds on what a kernel's
roundings may add.

Bounds of an attention output follow window_oracle: the result's own rounding u, P
rounded to bf16 (2^-8, for fp32 2^-24), the exponential's argument, n fp32 additions.
Over an 8-bit cache P times the value's scale is rounded to fp16 instead: 2^-11 of it, or
2^-25 where it is below fp16's normal numbers.  The kernel keeps the largest P sv of a row
above 1 in those units, so that what 2^-25 stands for is at most 2^-25 max(P sv) |code|, with
|code| <= 448 and n keys.  The queries become fp16 too: exact, but for elements below
2^-21 of their row's largest, which are off by at most 2^-32 of that."""
from __future__ import annotations

import numpy as np

import window_oracle as W

U32 = 2.0 ** -24


def e4m3_table():
    import torch
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)


def quantise(x):
    """Rows [..., d]: codes' values and scales by the definition (a loop over exponents would
    do the same: s is the smallest power of two >= 2^-100 with max|x| <= 448 s)."""
    import torch
    x = np.asarray(x, dtype=np.float64)
    top = np.abs(x).max(-1)
    fine = np.isfinite(x).all(-1)
    e = np.full(top.shape, -100)
    for i in range(-100, 122):
        e = np.where(fine & (top > 448 * 2.0 ** i), i + 1, e)
    s = 2.0 ** e.astype(np.float64)
    y = np.where(fine[..., None], x / s[..., None], 0.0)
    codes = torch.from_numpy(y).to(torch.float32).to(torch.float8_e4m3fn)   # y has at most 24 bits: one rounding
    return codes.float().numpy().astype(np.float64), np.where(fine, s, np.nan), codes


def slots_held(L, cap, sinks):
    """Positions that a cache of L appended ones holds, and their slots."""
    ring = cap - sinks
    p = [x for x in list(range(min(sinks, L))) + list(range(max(L - ring, sinks), L))]
    return np.array(p, dtype=np.int64), np.array([W.slot(x, cap, sinks) for x in p], dtype=np.int64)


def ancestors(parents, T):
    """[T, T]: which nodes a node descends from, itself among them; a parent that is not below
    its node counts as none."""
    a = np.eye(T, dtype=bool)
    for t in range(T):
        p = t - 1 if parents is None else int(parents[t])
        if 0 <= p < t:
            a[t] |= a[p]
    return a


def attention(q, k, v, scale, see, u, kv_scales=None):
    """One head, q [n, d] over k, v [m, d] where see [n, m]: O, LSE and bounds.  kv_scales: the
    scales of the values' first len(kv_scales) rows, which are 8-bit ones."""
    s = np.where(see, q @ k.T * scale, -np.inf)
    lse = np.full(len(q), -np.inf)
    some = see.any(-1)
    if some.any():
        m = s[some].max(-1)
        lse[some] = m + np.log(np.exp(s[some] - m[:, None]).sum(-1))
    p = np.where(see, np.exp(s - np.where(some, lse, 0.0)[:, None]), 0.0)
    vz = np.where(see.any(0)[:, None], v, 0.0)
    kz = np.where(see.any(0)[:, None], k, 0.0)
    o = p @ vz
    n = max(k.shape[0], 1)
    a = abs(scale) * (np.abs(q) @ np.abs(kz).T)
    ex = np.where(see, U32 * (q.shape[1] + 8) * (a + np.abs(np.where(some, lse, 0.0))[:, None]), 0.0)
    up = u if u > U32 else U32
    extra = 0.0
    if kv_scales is not None and u > U32:
        ex = ex + np.where(see, abs(scale) * 2.0 ** -32 * np.abs(q).max(-1, keepdims=True) * np.abs(kz).sum(-1)[None], 0.0)
        sv = np.concatenate([kv_scales, np.ones(len(k) - len(kv_scales))])
        extra = 2.0 ** -25 * 448 * n * (p * np.where(see, sv[None], 0.0)).max(-1, initial=0.0)[:, None]
    bo = u * np.abs(o) + (p * (up + 2 * ex + 2.0 ** -20 + n * U32)) @ np.abs(vz) + extra
    bl = (p * (2 * ex)).sum(-1) + 2.0 ** -20 + n * U32 + U32 * np.abs(np.where(some, lse, 0.0))
    return o, lse, bo, bl


def tree(q, k, v, kn, vn, lens, n_new, parents, cap, window, sinks, scale, u, v_scale=None):
    """q [B, Hq, T, d] over caches k, v [B, Hkv, cap, d] (their values) and the new rows kn, vn [B,
    Hkv, T, d]; parents [B, T] or None: O, LSE, bounds.  kn None: q is the newest cached token."""
    B, Hq, T, d = q.shape
    G = Hq // k.shape[1]
    o, bo = np.zeros(q.shape), np.zeros(q.shape)
    lse, bl = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3])
    for b in range(B):
        L = max(int(lens[b]), 0)
        held, slot = slots_held(L, cap, sinks)
        if kn is None:
            n, at, pos = 1, np.array([L - 1]), held
            own = np.zeros((1, 0), dtype=bool)
        else:
            n = min(max(int(n_new[b]), 0), T)
            line = ancestors(None if parents is None else parents[b], T)[:n, :n]
            at = L + line.sum(-1) - 1
            pos, own = np.concatenate([held, at]), line
        if n == 0 or len(pos) == 0:
            continue
        see = (pos[None] <= at[:, None]) & ((pos[None] > at[:, None] - window) | (pos[None] < sinks))
        see[:, len(held):] &= own
        for h in range(Hq):
            kk, vv = k[b, h // G][slot], v[b, h // G][slot]
            if kn is not None:
                kk, vv = np.concatenate([kk, kn[b, h // G, :n]]), np.concatenate([vv, vn[b, h // G, :n]])
            sv = None if v_scale is None else v_scale[b, h // G][slot]
            o[b, h, :n], lse[b, h, :n], bo[b, h, :n], bl[b, h, :n] = attention(q[b, h, :n], kk, vv, scale, see, u, sv)
    return o, lse, bo, bl
