"""Cases of the sliding-window attention family: rotary positions with several
axes, attention over a sliding window with a few first tokens that stay visible
(sinks), forward and backward, the rolling key/value cache of such a model and
the single-token attention that reads it.

`run` computes one pass, either in plain torch operations (`own` false) or
through this package's entry points (`own` true).  Tensors are [B, heads, N, d]
views of token-major [B, N, heads, d] memory, as a projection leaves them.

Definitions.  Query row i of sequence b has the position p = L_b - Q_b + i (Q_b
query rows, L_b keys; rows i >= Q_b are padding) and sees key j when
j <= p and (j > p - window or j < sinks).  A row that sees nothing has the
output 0 and the log-sum-exp -inf.  The rolling cache keeps position p in slot
p for p < sinks, else in slot sinks + (p - sinks) mod (capacity - sinks).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(name, op, dtype, B, Hq, Hkv, Nq, Nk, d, window=0, sinks=0, ragged=False, axes=1, capacity=0, inverse=False,
          ladder="shared", pairing="halves"):
    c = dict(op=op, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, Nq=Nq, Nk=Nk, d=d, window=window, sinks=sinks, ragged=ragged,
             axes=axes, capacity=capacity, inverse=inverse, ladder=ladder, pairing=pairing)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decoding step of 16 requests: the rotation of one query and one key per head
        _case("rope_token", "rope", "bf16", 16, 16, 4, 1, 1, 128),
        # gradients of the rotation over video: 16 frames of a 20x20 map, (time, row, column) positions
        _case("rope_video_grad", "rope", "bf16", 2, 16, 8, 6400, 6400, 64, axes=3, inverse=True),
        # a padded batch of short sequences of different lengths
        _case("fwd_short_ragged", "fwd", "bf16", 8, 8, 2, 400, 400, 64, window=128, sinks=4, ragged=True),
        # one long prompt: prefill of 16K tokens
        _case("fwd_long", "fwd", "bf16", 1, 16, 4, 16384, 16384, 128, window=1024, sinks=4),
        # 32-bit storage, one head per key head, an odd window
        _case("fwd_f32", "fwd", "f32", 2, 4, 4, 1600, 1600, 32, window=333, sinks=1),
        # a training step's gradients for the padded batch of short sequences
        _case("bwd_short_ragged", "bwd", "bf16", 8, 8, 2, 400, 400, 64, window=128, sinks=4, ragged=True),
        # a training step's gradients at a long context
        _case("bwd_long", "bwd", "bf16", 1, 16, 4, 8192, 8192, 128, window=1024, sinks=4),
        # 32-bit gradients
        _case("bwd_f32", "bwd", "f32", 2, 4, 4, 1600, 1600, 32, window=333, sinks=1),
        # prompts of 4 requests written into their caches, keys rotated on the way
        _case("append_prompt", "append", "bf16", 4, 0, 8, 2048, 0, 128, window=1024, sinks=4, capacity=1028),
        # the newest token of 64 requests, behind different numbers of earlier ones
        _case("append_token", "append", "bf16", 64, 0, 8, 1, 0, 128, window=1024, sinks=4, capacity=1028, ragged=True),
        # one request's next token
        _case("decode_one", "decode", "bf16", 1, 16, 4, 1, 2000, 128, window=1024, sinks=4, capacity=1028),
        # 64 requests' next tokens, most of them with full windows
        _case("decode_batch", "decode", "bf16", 64, 32, 8, 1, 9000, 128, window=4096, sinks=4, capacity=4100,
              ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "fwd", "fwd", "bwd", "bwd", "append", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 7, 8])
    B = _log_int(rng, 1, 16)
    sinks = rng.choice([0, 1, 4, 17, 64])
    ragged = rng.random() < 0.5
    if op == "rope":
        N = _log_int(rng, 1, 8192)
        B = max(1, min(B, 4096 * 16 // (N * Hkv)))
        axes = rng.choice([1, 2, 3])
        return _case("", op, dtype, B, Hkv * G, Hkv, N, N, d, axes=axes, inverse=rng.random() < 0.5,
                     ladder=rng.choice(["shared", "per_axis"]), pairing=rng.choice(["halves", "interleaved"]))
    if op in ("fwd", "bwd"):
        # a gradient with a single visible key is zero but for rounding: two at least
        least = 2 if op == "bwd" else 1
        Nk = _log_int(rng, least, 4096 if dtype == "bf16" else 1500)
        # whole sequences, the last rows of a longer context, or more rows than keys (the first see nothing)
        Nq = rng.choice([Nk, Nk, Nk, Nk, _log_int(rng, 1, Nk), Nk + _log_int(rng, 1, 200)])
        B = max(1, min(B, 8, (1 << 25) // (Nq * Nk * Hkv * G)))
        window = _log_int(rng, least, max(least, min(Nk + 100, 2048)))
        return _case("", op, dtype, B, Hkv * G, Hkv, Nq, Nk, d, window=window, sinks=sinks, ragged=ragged)
    window = _log_int(rng, 1, 4096)
    slack = rng.choice([0, 0, 13])
    capacity = sinks + window + slack
    if op == "append":
        T = _log_int(rng, 1, 4096)
        B = max(1, min(B, (1 << 15) // T))
        return _case("", op, dtype, B, 0, Hkv, T, 0, d, window=window, sinks=sinks, capacity=capacity, ragged=ragged)
    return _case("", op, dtype, B * 2, Hkv * G, Hkv, 1, _log_int(rng, 1, 20000), d, window=window, sinks=sinks,
                 capacity=capacity, ragged=ragged)


def _spread(n, B, ragged):
    """Lengths of the B sequences of a batch: all n, or falling evenly from n to about n / 2."""
    return [max(1, n - (b * n) // (2 * B)) if ragged else n for b in range(B)]


def _sections(c):
    """Pairs of every axis: the time axis gets what the others leave."""
    pairs = c["d"] // 2
    rest = [pairs * 3 // 8, pairs * 3 // 8] if c["axes"] == 3 else [pairs // 2] if c["axes"] == 2 else []
    return [pairs - sum(rest)] + rest


THETA = 10000.0


def _turns(c):
    """(inverse frequency in 64 bits, axis) of every pair."""
    sec = _sections(c)
    axis = np.repeat(np.arange(len(sec)), sec)
    if c["ladder"] == "shared":
        e = np.arange(sum(sec)) / sum(sec)
    else:
        e = np.concatenate([np.arange(s) / s for s in sec])
    return THETA ** -e, axis


def _tokens(shape, dtype, g):
    """A [B, heads, N, d] view of token-major memory."""
    B, H, N, d = shape
    return torch.randn((B, N, H, d), generator=g, device="cuda", dtype=torch.float32).to(dtype).transpose(1, 2)


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    t, B, d = DTYPES[c["dtype"]], c["B"], c["d"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": c, "scale": 1.0 / math.sqrt(d)}
    if c["op"] in ("rope", "append"):
        inv, axis = _turns(c)
        s["inv_freq"] = torch.tensor(inv, dtype=torch.float64, device="cuda")
        s["axis"] = torch.tensor(axis, dtype=torch.int64, device="cuda")
    if c["op"] == "rope":
        s["q"] = _tokens((B, c["Hq"], c["Nq"], d), t, g)
        s["k"] = _tokens((B, c["Hkv"], c["Nk"], d), t, g)
        N = c["Nq"]
        first = torch.randint(0, 100000, (B, 1), generator=g, device="cuda")
        n = torch.arange(N, device="cuda")
        if c["axes"] == 1:
            pos = (first + n)[None]
        else:  # frames of a map 20 wide (and 20 high), frame after frame
            per = [first + n // 400, (n // 20 % 20).expand(B, N), (n % 20).expand(B, N)]
            pos = torch.stack(per if c["axes"] == 3 else per[1:])
        s["pos"] = pos.to(torch.int32).contiguous()
    elif c["op"] in ("fwd", "bwd"):
        s["q"] = _tokens((B, c["Hq"], c["Nq"], d), t, g)
        s["k"] = _tokens((B, c["Hkv"], c["Nk"], d), t, g)
        s["v"] = _tokens((B, c["Hkv"], c["Nk"], d), t, g)
        s["q_lens"], s["kv_lens"] = ints(_spread(c["Nq"], B, c["ragged"])), ints(_spread(c["Nk"], B, c["ragged"]))
        if c["op"] == "bwd":
            s["o"], s["lse"] = _plain_fwd(s)
            s["do"] = _tokens((B, c["Hq"], c["Nq"], d), t, g)
    else:
        shape = (B, c["Hkv"], c["capacity"], d)
        s["k_cache"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(t)
        s["v_cache"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(t)
        if c["op"] == "append":
            s["k"] = _tokens((B, c["Hkv"], c["Nq"], d), t, g)
            s["v"] = _tokens((B, c["Hkv"], c["Nq"], d), t, g)
            start = torch.randint(0, 20000, (B,), generator=g, device="cuda") * int(c["ragged"])
            s["start"] = start.to(torch.int32)
            s["n_new"] = ints(_spread(c["Nq"], B, c["ragged"]))
            s["pos"] = (start[:, None] + torch.arange(c["Nq"], device="cuda"))[None].to(torch.int32).contiguous()
        else:
            s["q"] = _tokens((B, c["Hq"], 1, d), t, g)
            s["lens"] = ints(_spread(c["Nk"], B, c["ragged"]))
    if own:  # the handles that a program makes once and keeps
        from self_attention_backward_gb300 import binding
        s["binding"] = binding
        if "inv_freq" in s:
            ladder = binding.PSA_ROPE_SHARED if c["ladder"] == "shared" else binding.PSA_ROPE_PER_AXIS
            s["plan"] = binding.RopePlan(d, _sections(c), theta=THETA, ladder=ladder,
                                         interleaved=c["pairing"] == "interleaved")
        if "k_cache" in s:
            s["cache"] = binding.WinCache(s["k_cache"], s["v_cache"], c["window"], c["sinks"])
        if c["op"] == "bwd":
            s["workspace"] = binding.BwdWorkspace()
    return s


# ----------------------------------------------------------------- plain forms
def _rotate(x, s, inverse):
    """Rotary positions: x [B, H, N, d] in 32 bits, angles in 64."""
    c = s["case"]
    angle = s["pos"].double()[s["axis"]].permute(1, 2, 0) * s["inv_freq"]      # [B, N, pairs]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    sin = -sin if inverse else sin
    h = c["d"] // 2
    if c["pairing"] == "halves":
        a, b = x[..., :h].float(), x[..., h:].float()
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2].float(), x[..., 1::2].float()
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _visible(s):
    """[B, 1, 1, Nq, Nk]: which keys a query row sees."""
    c = s["case"]
    ql, kl = s["q_lens"].long()[:, None, None], s["kv_lens"].long()[:, None, None]
    i = torch.arange(c["Nq"], device="cuda")[None, :, None]
    j = torch.arange(c["Nk"], device="cuda")[None, None, :]
    p = kl - ql + i
    return ((i < ql) & (j <= p) & ((j > p - c["window"]) | (j < c["sinks"])))[:, None, None]


def _grouped(x, c):
    """[B, Hq, N, d] -> [B, Hkv, G, N, d] in 32 bits."""
    return x.float().unflatten(1, (c["Hkv"], -1))


def _plain_fwd(s):
    c, t = s["case"], s["q"].dtype
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    x = (_grouped(s["q"], c) @ k.transpose(-1, -2)) * s["scale"]
    x = x.masked_fill_(~_visible(s), -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = x.sub_(m).exp_()
    l = e.sum(-1, keepdim=True)
    o = (e @ v) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log(l))[..., 0].flatten(1, 2)
    return o.flatten(1, 2).to(t), lse


def _plain_bwd(s):
    c, t, scale = s["case"], s["q"].dtype, s["scale"]
    q, do, o = _grouped(s["q"], c), _grouped(s["do"], c), _grouped(s["o"], c)
    k, v = s["k"].float()[:, :, None], s["v"].float()[:, :, None]
    lse = s["lse"].unflatten(1, (c["Hkv"], -1))[..., None]
    lse = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)
    p = (q @ k.transpose(-1, -2)) * scale
    p = p.masked_fill_(~_visible(s), -math.inf).sub_(lse).exp_()
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k) * scale
    dk = (ds.transpose(-1, -2) @ q).sum(2) * scale
    dv = (p.transpose(-1, -2) @ do).sum(2)
    return dq.flatten(1, 2).to(t), dk.to(t), dv.to(t)


def _plain_append(s):
    """Of the tokens that share a slot only the newest is written."""
    c = s["case"]
    ring = c["capacity"] - c["sinks"]
    start, n = s["start"].long()[:, None], s["n_new"].long()[:, None]
    t = torch.arange(c["Nq"], device="cuda")[None]
    p = start + t
    b, t = ((t < n) & ((p < c["sinks"]) | (p >= start + n - ring))).nonzero(as_tuple=True)
    p = p[b, t]
    slot = torch.where(p < c["sinks"], p, c["sinks"] + (p - c["sinks"]) % ring)
    s["k_cache"][b, :, slot] = _rotate(s["k"], s, False).to(s["k"].dtype)[b, :, t]
    s["v_cache"][b, :, slot] = s["v"][b, :, t]
    return s["k_cache"], s["v_cache"]


def _plain_decode(s):
    c = s["case"]
    ring = c["capacity"] - c["sinks"]
    L = s["lens"].long()[:, None]
    slot = torch.arange(c["capacity"], device="cuda")[None]
    newest = slot + torch.div(L - 1 - slot, ring, rounding_mode="floor") * ring
    seen = torch.where(slot < c["sinks"], slot < L, (newest >= slot) & (newest > L - 1 - c["window"]))
    q = _grouped(s["q"], c)
    x = (q @ s["k_cache"].float()[:, :, None].transpose(-1, -2)) * s["scale"]
    x = x.masked_fill_(~seen[:, None, None, None], -math.inf)
    e = (x - x.amax(-1, keepdim=True)).exp_()
    o = (e @ s["v_cache"].float()[:, :, None]) / e.sum(-1, keepdim=True)
    return o.flatten(1, 2)[:, :, 0].to(s["q"].dtype)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        B = s["binding"]
        if op == "rope":
            return B.rope(s["plan"], s["q"], s["pos"], k=s["k"], inverse=c["inverse"])
        if op == "append":
            s["cache"].append(s["k"], s["v"], s["start"], n_new=s["n_new"], plan=s["plan"], pos=s["pos"])
            return s["k_cache"], s["v_cache"]
        if op == "decode":
            return s["cache"].decode(s["q"][:, :, 0], s["lens"], s["scale"])
        lens = dict(q_lens=s["q_lens"], kv_lens=s["kv_lens"]) if c["ragged"] else {}
        if op == "fwd":
            return B.win_attn_fwd(s["q"], s["k"], s["v"], s["scale"], c["window"], c["sinks"], **lens)
        return B.win_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["scale"], c["window"], c["sinks"],
                              workspace=s["workspace"], **lens)
    if op == "rope":
        t = s["q"].dtype
        return _rotate(s["q"], s, c["inverse"]).to(t), _rotate(s["k"], s, c["inverse"]).to(t)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "append": _plain_append, "decode": _plain_decode}[op](s)


# ----------------------------------------------------------------- floors
def _seen_pairs(c):
    """Visible (query, key) pairs of one head, summed over the batch, and the keys that some row sees."""
    pairs, keys = 0, 0
    for ql, kl in zip(_spread(c["Nq"], c["B"], c["ragged"]), _spread(c["Nk"], c["B"], c["ragged"])):
        p = np.arange(max(0, kl - ql), kl, dtype=np.int64)
        low = np.maximum(p + 1 - c["window"], 0)
        pairs += int((p + 1 - low + np.minimum(low, c["sinks"])).sum())
        if p.size:
            keys += int(kl - low[0] + min(low[0], c["sinks"]))
    return pairs, keys


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    d, B = c["d"], c["B"]
    if c["op"] == "rope":
        n = B * c["Nq"] * (c["Hq"] + c["Hkv"])
        return {"bytes": 2 * n * d * e + 4 * c["axes"] * B * c["Nq"], "flops": 3 * n * d}
    if c["op"] == "append":
        ring = c["capacity"] - c["sinks"]
        n = sum(min(t, c["sinks"] + ring) for t in _spread(c["Nq"], B, c["ragged"])) * c["Hkv"]
        return {"bytes": 4 * n * d * e, "flops": 3 * n * d}
    if c["op"] == "decode":
        n = sum(min(t, c["sinks"] + c["window"]) for t in _spread(c["Nk"], B, c["ragged"]))
        return {"bytes": 2 * n * c["Hkv"] * d * e + 2 * B * c["Hq"] * d * e, "flops": 4 * n * c["Hq"] * d}
    pairs, keys = _seen_pairs(c)
    rows = sum(_spread(c["Nq"], B, c["ragged"])) * c["Hq"]
    kv = keys * c["Hkv"] * d * e
    if c["op"] == "fwd":
        return {"bytes": 2 * kv + 2 * rows * d * e + 4 * rows, "flops": 4 * pairs * c["Hq"] * d}
    return {"bytes": 4 * kv + 4 * rows * d * e + 4 * rows, "flops": 10 * pairs * c["Hq"] * d}


# ----------------------------------------------------------------- the definitions in 64 bits
def _exact_rotation(x, pos, c, inverse):
    """One rotation matrix entry after the other: complex numbers times exp(i angle)."""
    inv, axis = _turns(c)
    ids = pos.double()
    ang = torch.stack([ids[a] * f for a, f in zip(axis.tolist(), inv.tolist())], -1)[:, None]   # [B, 1, N, pairs]
    z = x.double()
    h = c["d"] // 2
    z = torch.complex(z[..., :h], z[..., h:]) if c["pairing"] == "halves" else torch.view_as_complex(
        z.reshape(*z.shape[:-1], h, 2).contiguous())
    z = z * torch.polar(torch.ones_like(ang), -ang if inverse else ang)
    return torch.cat([z.real, z.imag], -1) if c["pairing"] == "halves" else torch.view_as_real(z).flatten(-2)


def _exact_attention(s, grad):
    c, scale = s["case"], s["scale"]
    B, G, d = c["B"], c["Hq"] // c["Hkv"], c["d"]
    f8 = dict(dtype=torch.float64, device="cuda")
    o = torch.zeros((B, c["Hq"], c["Nq"], d), **f8)
    lse = torch.full((B, c["Hq"], c["Nq"]), -math.inf, **f8)
    dq, dk, dv = torch.zeros_like(o), torch.zeros((B, c["Hkv"], c["Nk"], d), **f8), torch.zeros(
        (B, c["Hkv"], c["Nk"], d), **f8)
    step = 1024
    for b, (ql, kl) in enumerate(zip(_spread(c["Nq"], B, c["ragged"]), _spread(c["Nk"], B, c["ragged"]))):
        for i0 in range(0, ql, step):
            i1 = min(ql, i0 + step)
            p0, p1 = kl - ql + i0, kl - ql + i1 - 1
            if p1 < 0:
                continue
            low = max(0, p0 - c["window"] + 1)
            idx = torch.cat([torch.arange(min(c["sinks"], low), device="cuda"), torch.arange(low, p1 + 1, device="cuda")])
            p = torch.arange(p0, p1 + 1, device="cuda")[:, None]
            hidden = (idx[None] > p) | ((idx[None] <= p - c["window"]) & (idx[None] >= c["sinks"]))
            for h in range(c["Hq"]):
                kk, vv = s["k"][b, h // G, idx].double(), s["v"][b, h // G, idx].double()
                qq = s["q"][b, h, i0:i1].double()
                x = torch.einsum("id,jd->ij", qq, kk) * scale
                x[hidden] = -math.inf
                if not grad:
                    some = ~hidden.all(-1)
                    lse[b, h, i0:i1] = torch.logsumexp(x, -1)
                    o[b, h, i0:i1][some] = torch.softmax(x[some], -1) @ vv
                    continue
                st = s["lse"][b, h, i0:i1].double()[:, None]
                pr = torch.where(hidden, 0.0, torch.exp(x - torch.where(torch.isinf(st), 0.0, st)))
                g = s["do"][b, h, i0:i1].double()
                ds = pr * (g @ vv.T - (g * s["o"][b, h, i0:i1].double()).sum(-1, keepdim=True))
                dq[b, h, i0:i1] = scale * (ds @ kk)
                dk[b, h // G].index_add_(0, idx, scale * (ds.T @ qq))
                dv[b, h // G].index_add_(0, idx, pr.T @ g)
    return (dq, dk, dv) if grad else (o, lse)


def _exact_append(s):
    """For every slot of every sequence, the newest token that lands in it, or what it held."""
    c = s["case"]
    ring = c["capacity"] - c["sinks"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    k, v = _exact_rotation(s["k"], s["pos"], c, False), s["v"].double()
    for b, (a, n) in enumerate(zip(s["start"].tolist(), s["n_new"].tolist())):
        holds = {}
        for p in range(a, a + n):
            holds[p if p < c["sinks"] else c["sinks"] + (p - c["sinks"]) % ring] = p - a
        slot, t = torch.tensor(list(holds)), torch.tensor(list(holds.values()))
        kc[b][:, slot] = k[b][:, t]
        vc[b][:, slot] = v[b][:, t]
    return kc, vc


def _exact_decode(s):
    c = s["case"]
    ring, G = c["capacity"] - c["sinks"], c["Hq"] // c["Hkv"]
    o = torch.zeros((c["B"], c["Hq"], c["d"]), dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        p = torch.arange(L, device="cuda")
        p = p[(p < c["sinks"]) | (p > L - 1 - c["window"])]
        slot = torch.where(p < c["sinks"], p, c["sinks"] + (p - c["sinks"]) % ring)
        for h in range(c["Hkv"]):
            x = torch.einsum("gd,jd->gj", s["q"][b, h * G:(h + 1) * G, 0].double(), s["k_cache"][b, h, slot].double())
            o[b, h * G:(h + 1) * G] = torch.softmax(x * s["scale"], -1) @ s["v_cache"][b, h, slot].double()
    return o


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return tuple(_exact_rotation(s[x], s["pos"], case, case["inverse"]) for x in ("q", "k"))
    if op == "append":
        return _exact_append(s)
    if op == "decode":
        return _exact_decode(s)
    return _exact_attention(s, op == "bwd")
