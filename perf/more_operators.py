"""Cases of serving with drafted tokens over a rolling key/value cache: the
attention of a tree (or a run) of new tokens over the cache, the accepted path
written into it, and the same cache held in 8 bits, quantised as it is written,
read back, and attended to by single tokens and by trees.

`run` computes one pass, either in plain torch operations (`own` false) or
through this package's entry points (`own` true).  New tokens are [B, heads, T, d]
views of token-major [B, T, heads, d] memory, as a projection leaves them.

Definitions.  The cache keeps position p in slot p for p < sinks, else in slot
sinks + (p - sinks) mod (capacity - sinks).  A single token at position lens - 1
sees the positions j < lens with j < sinks or j >= lens - window.  Node t of a
tree has the parent parents[t] < t, or -1 for none; its position is p = lens +
(number of its ancestors).  It sees the cached positions j < lens with j < sinks
or j > p - window, and of its ancestors and itself those whose position is below
sinks or above p - window.  Rows past n_new are padding: their output is 0.
An 8-bit row x is codes times a scale: the scale is the smallest power of two s
with max|x| <= 448 s, the codes are x / s rounded to e4m3 (to nearest, ties to even).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
THETA = 10000.0


def _case(name, op, dtype, B, Hq, Hkv, T, L, d, window, sinks, capacity=0, bits8=False, ragged=False, tree=True, R=0):
    """T new tokens behind L cached ones; R: the longest accepted path."""
    c = dict(op=op, dtype=dtype, B=B, Hq=Hq, Hkv=Hkv, T=T, L=L, d=d, window=window, sinks=sinks,
             capacity=capacity or sinks + window, bits8=bits8, ragged=ragged, tree=tree, R=R)
    return dict(c, name=name) if name else c


def listed():
    return [
        # the newest token of 64 requests, rotated, quantised and read back
        _case("store_token", "store", "bf16", 64, 0, 8, 1, 5000, 128, 4096, 4, bits8=True, ragged=True),
        # prompts of 4 requests into their 8-bit caches, read back for the prompt's own attention
        _case("store_prompt", "store", "bf16", 4, 0, 8, 2048, 0, 128, 4096, 4, bits8=True),
        # the accepted paths of 16 requests' trees of 64 nodes
        _case("accept", "accept", "bf16", 16, 0, 8, 64, 5000, 128, 1024, 4, ragged=True, R=8),
        # the same into 8-bit caches of a 32-bit model
        _case("accept_8bit", "accept", "f32", 64, 0, 4, 32, 5000, 64, 1024, 4, bits8=True, ragged=True, R=6),
        # one request's next token
        _case("decode_one_8bit", "decode", "bf16", 1, 16, 4, 1, 2000, 128, 1024, 4, bits8=True),
        # 64 requests' next tokens, all of them with full windows
        _case("decode_batch_8bit", "decode", "bf16", 64, 32, 8, 1, 9000, 128, 4096, 4, bits8=True, ragged=True),
        # one request's tree of 26 drafted tokens
        _case("tree_one", "tree", "bf16", 1, 16, 4, 26, 6000, 128, 4096, 4),
        # 16 requests' trees of up to 64 drafted tokens
        _case("tree_batch", "tree", "bf16", 16, 32, 8, 64, 9000, 128, 4096, 4, ragged=True),
        # the next 256 tokens of 4 long prompts: a run of tokens over a cache that keeps everything
        _case("run_long", "tree", "bf16", 4, 16, 4, 256, 30000, 128, 32764, 4, tree=False),
        # a small 32-bit model, odd sizes
        _case("tree_f32", "tree", "f32", 2, 4, 4, 17, 1600, 32, 333, 1),
        # one request's tree over a long 8-bit cache
        _case("tree_one_8bit", "tree", "bf16", 1, 16, 4, 32, 20000, 128, 32764, 4, bits8=True),
        # 32 requests' trees of up to 16 drafted tokens over 8-bit caches
        _case("tree_batch_8bit", "tree", "bf16", 32, 32, 8, 16, 9000, 128, 4096, 4, bits8=True, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "accept", "decode", "tree", "tree", "tree", "tree"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 4, 7, 8])
    sinks = rng.choice([0, 1, 4, 17, 64])
    window = _log_int(rng, 1, 16384)
    capacity = sinks + window + rng.choice([0, 0, 13])
    ragged = rng.random() < 0.5
    L = _log_int(rng, 1, 20000)
    kw = dict(window=window, sinks=sinks, capacity=capacity, ragged=ragged)
    if op == "store":
        T = _log_int(rng, 1, 4096)
        B = max(1, min(_log_int(rng, 1, 64), (1 << 14) // T, (1 << 24) // (capacity * Hkv * d) + 1))
        return _case("", op, dtype, B, 0, Hkv, T, rng.choice([0, L]), d, bits8=True, **kw)
    bits8 = op == "decode" or rng.random() < 0.5
    T = 1 if op == "decode" else _log_int(rng, 1, 256)
    n = min(L, sinks + window)
    B = max(1, min(_log_int(rng, 1, 64), (1 << 27) // (capacity * Hkv * d), (1 << 27) // (n * T * Hkv * G)))
    if op == "accept":
        return _case("", op, dtype, B, 0, Hkv, T, L, d, bits8=bits8, R=_log_int(rng, 1, min(T, 16)), **kw)
    return _case("", op, dtype, B, Hkv * G, Hkv, T, L, d, bits8=bits8, tree=rng.random() < 0.7, **kw)


def _spread(n, B, ragged):
    """B numbers: all n, or falling evenly from n to about n / 2."""
    return [max(min(n, 1), n - (b * n) // (2 * B)) if ragged else n for b in range(B)]


def _tokens(shape, dtype, g):
    """A [B, heads, N, d] view of token-major memory."""
    B, H, N, d = shape
    return torch.randn((B, N, H, d), generator=g, device="cuda", dtype=torch.float32).to(dtype).transpose(1, 2)


def _quantise(x):
    """32-bit rows -> e4m3 codes and 32-bit scales."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = e - 9 + (m > 0.875).to(e.dtype)                      # 448 = 0.875 2^9
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), torch.ldexp(torch.ones_like(m), e)


def _lens(c):
    """Cached positions of every sequence."""
    return _spread(c["L"], c["B"], c["ragged"])


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    t, B, T, d = DTYPES[c["dtype"]], c["B"], c["T"], c["d"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": c, "scale": 1.0 / math.sqrt(d), "lens": ints(_lens(c)), "n_new": ints(_spread(T, B, c["ragged"]))}
    shape = (B, c["Hkv"], c["capacity"], d)
    for x in ("k", "v"):
        full = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(t)
        if c["bits8"]:
            # heads and tokens of different sizes, as keys and values have them
            full = full.float().mul_(torch.exp(0.5 * torch.randn((*shape[:3], 1), generator=g, device="cuda")))
            s[x + "_cache"], s[x + "_scale"] = _quantise(full)
        else:
            s[x + "_cache"], s[x + "_scale"] = full, None
    if c["op"] == "decode":
        s["q"] = _tokens((B, c["Hq"], 1, d), t, g)
    else:
        s["k"], s["v"] = _tokens((B, c["Hkv"], T, d), t, g), _tokens((B, c["Hkv"], T, d), t, g)
    if c["op"] == "store":
        s["after"] = s["lens"] + s["n_new"]
        s["pos"] = (s["lens"][:, None] + torch.arange(T, device="cuda", dtype=torch.int32))[None].contiguous()
        s["inv_freq"] = torch.tensor(THETA ** -(np.arange(d // 2) / (d // 2)), dtype=torch.float64, device="cuda")
    if c["op"] == "accept":
        # a path down the tree: growing node numbers
        step = 1 + torch.randint(0, max(1, T // c["R"]), (B, c["R"]), generator=g, device="cuda")
        s["path"] = (step.cumsum(1) - 1).to(torch.int32).contiguous()
        s["n_new"] = ints(_spread(c["R"], B, c["ragged"]))
        s["after"] = s["lens"] + s["n_new"]
    if c["op"] == "tree":
        s["q"] = _tokens((B, c["Hq"], T, d), t, g)
        n = torch.arange(T, device="cuda")
        back = torch.randint(1, 9, (B, T), generator=g, device="cuda")      # a few branches at every depth
        s["parents"] = torch.where(n == 0, -1, (n - back).clamp(min=0)).to(torch.int32).contiguous() if c["tree"] else None
    if own:  # the handles that a program makes once and keeps
        from self_attention_backward_gb300 import binding
        s["cache"] = binding.WinCache(s["k_cache"], s["v_cache"], c["window"], c["sinks"], s["k_scale"], s["v_scale"])
        if c["op"] == "store":
            s["plan"] = binding.RopePlan(d, (d // 2,), theta=THETA)
    return s


# ----------------------------------------------------------------- plain forms
def _rotate(x, s):
    """Rotary positions, pairs in halves: x [B, H, T, d] in 32 bits, angles in 64."""
    h = s["case"]["d"] // 2
    angle = s["pos"][0].double()[..., None] * s["inv_freq"]                   # [B, T, pairs]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = x[..., :h].float(), x[..., h:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _slot(p, c):
    return torch.where(p < c["sinks"], p, c["sinks"] + (p - c["sinks"]) % (c["capacity"] - c["sinks"]))


def _write(s, k, v, n):
    """Rows [B, H, N, d] to the positions lens .. lens + n - 1; of the rows that share a slot only the newest."""
    c = s["case"]
    start, n = s["lens"].long()[:, None], n.long()[:, None]
    t = torch.arange(k.shape[2], device="cuda")[None]
    p = start + t
    b, t = ((t < n) & ((p < c["sinks"]) | (p >= start + n - (c["capacity"] - c["sinks"])))).nonzero(as_tuple=True)
    slot = _slot(p[b, t], c)
    if c["bits8"]:
        (k, ks), (v, vs) = _quantise(k.float()), _quantise(v.float())
        s["k_scale"][b, :, slot], s["v_scale"][b, :, slot] = ks[b, :, t], vs[b, :, t]
        # torch indexes bytes, not e4m3
        s["k_cache"].view(torch.uint8)[b, :, slot] = k.view(torch.uint8)[b, :, t]
        s["v_cache"].view(torch.uint8)[b, :, slot] = v.view(torch.uint8)[b, :, t]
    else:
        s["k_cache"][b, :, slot], s["v_cache"][b, :, slot] = k.to(s["k"].dtype)[b, :, t], v.to(s["v"].dtype)[b, :, t]


def _values(x, scale):
    return x.float() if scale is None else x.float() * scale[..., None]


def _read(s, N):
    """The N positions from lens on, 0 where the cache does not hold them, as bf16."""
    c = s["case"]
    p = s["lens"].long()[:, None] + torch.arange(N, device="cuda")[None]
    after = s["after"].long()[:, None]
    held = (p < after) & ((p < c["sinks"]) | (p >= after - (c["capacity"] - c["sinks"])))
    b, slot = torch.arange(c["B"], device="cuda")[:, None], _slot(p, c)

    def rows(x, scale):
        codes = x.view(torch.uint8)[b, :, slot].view(x.dtype) if scale is not None else x[b, :, slot]
        y = _values(codes, None if scale is None else scale[b, :, slot])
        return torch.where(held[..., None, None], y, 0.0).transpose(1, 2).to(torch.bfloat16)

    return rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])


def _seen_slots(s, L, ahead):
    """[B, ahead's T, capacity]: which slots a token `ahead` positions behind the newest cached one sees."""
    c = s["case"]
    ring = c["capacity"] - c["sinks"]
    slot = torch.arange(c["capacity"], device="cuda")[None]
    newest = slot + torch.div(L - 1 - slot, ring, rounding_mode="floor") * ring
    seen = (newest >= slot)[:, None] & (newest[:, None] > (L - 1)[..., None] + ahead[..., None] - c["window"])
    return torch.where(slot < c["sinks"], (slot < L)[:, None], seen)


def _grouped(x, c):
    """[B, Hq, N, d] -> [B, Hkv, G, N, d] in 32 bits."""
    return x.float().unflatten(1, (c["Hkv"], -1))


def _plain_decode(s):
    c = s["case"]
    L = s["lens"].long()[:, None]
    seen = _seen_slots(s, L, torch.zeros_like(L))[:, None, None]
    k, v = _values(s["k_cache"], s["k_scale"])[:, :, None], _values(s["v_cache"], s["v_scale"])[:, :, None]
    x = (_grouped(s["q"], c) @ k.transpose(-1, -2)) * s["scale"]
    x = x.masked_fill_(~seen, -math.inf)
    e = (x - x.amax(-1, keepdim=True)).exp_()
    o = (e @ v) / e.sum(-1, keepdim=True)
    return o.flatten(1, 2)[:, :, 0].to(s["q"].dtype)


def _ancestors(s):
    """[B, T, T] truth values: which nodes a node descends from, itself among them."""
    c = s["case"]
    n = torch.arange(c["T"], device="cuda")
    if s["parents"] is None:
        return (n[None, :] <= n[:, None]).expand(c["B"], -1, -1)
    step = (s["parents"][..., None] == n).float()            # 1 + step + step^2 + ... = 1 / (1 - step), of 0s and 1s
    one = torch.eye(c["T"], device="cuda").expand_as(step)
    return torch.linalg.solve_triangular(one - step, one, upper=False, unitriangular=True) > 0.5


def _plain_tree(s):
    c = s["case"]
    B, T, H, cap = c["B"], c["T"], c["Hkv"], c["capacity"]
    up = _ancestors(s)
    depth = up.sum(-1) - 1                                    # [B, T]
    L = s["lens"].long()[:, None]
    p = L + depth
    up = up & ((p[:, None, :] > p[..., None] - c["window"]) | (p < c["sinks"])[:, None, :])
    seen = torch.cat([_seen_slots(s, L, depth + 1), up], -1)[:, None, None]   # [B, 1, 1, T, capacity + T]
    k = torch.cat([_values(s["k_cache"], s["k_scale"]), s["k"].float()], 2)
    v = torch.cat([_values(s["v_cache"], s["v_scale"]), s["v"].float()], 2)
    q = _grouped(s["q"], c).flatten(2, 3)                     # [B, H, G T, d]
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(B, H, -1, T, cap + T)
    x = x.masked_fill_(~seen, -math.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x.flatten(2, 3) @ v).view(B, H, -1, T, c["d"]) / l
    real = torch.arange(T, device="cuda") < s["n_new"][:, None]
    return torch.where(real[:, None, None, :, None], o, 0.0).flatten(1, 2).to(s["q"].dtype)


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        cache = s["cache"]
        if op == "store":
            cache.append(s["k"], s["v"], s["lens"], n_new=s["n_new"], plan=s["plan"], pos=s["pos"])
            return cache.read(s["lens"], c["T"], s["after"], dtype=torch.bfloat16)
        if op == "accept":
            cache.append(s["k"], s["v"], s["lens"], n_new=s["n_new"], rows=s["path"])
            if c["bits8"]:
                return cache.read(s["lens"], c["R"], s["after"], dtype=torch.bfloat16)
            return s["k_cache"], s["v_cache"]
        if op == "decode":
            return cache.decode(s["q"][:, :, 0], s["lens"], s["scale"])
        return cache.tree(s["q"], s["k"], s["v"], s["lens"], s["scale"], parents=s["parents"],
                          n_new=s["n_new"] if c["ragged"] else None)
    if op == "store":
        _write(s, _rotate(s["k"], s), s["v"], s["n_new"])
        return _read(s, c["T"])
    if op == "accept":
        at = s["path"].long()[:, None, :, None].expand(-1, c["Hkv"], -1, c["d"])
        _write(s, s["k"].gather(2, at), s["v"].gather(2, at), s["n_new"])
        return _read(s, c["R"]) if c["bits8"] else (s["k_cache"], s["v_cache"])
    return _plain_decode(s) if op == "decode" else _plain_tree(s)


# ----------------------------------------------------------------- floors
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    d, B, H, T = c["d"], c["B"], c["Hkv"], c["T"]
    held = d + 4 if c["bits8"] else d * e                     # bytes of a cached row
    ring = c["capacity"] - c["sinks"]
    if c["op"] == "store":                                    # rows read, written, read back as bf16
        n = sum(min(t, c["sinks"] + ring) for t in _spread(T, B, c["ragged"])) * H
        return {"bytes": 2 * n * (d * e + 2 * held) + 2 * B * T * H * 2 * d, "flops": 3 * n * d}
    if c["op"] == "accept":
        n = sum(min(t, c["sinks"] + ring) for t in _spread(c["R"], B, c["ragged"])) * H
        back = 2 * n * held + 2 * B * c["R"] * H * 2 * d if c["bits8"] else 0
        return {"bytes": 2 * n * (d * e + held) + back, "flops": n * d}
    seen = [min(t, c["sinks"] + c["window"]) for t in _lens(c)]
    if c["op"] == "decode":
        n = sum(seen)
        return {"bytes": 2 * n * H * held + 2 * B * c["Hq"] * d * e, "flops": 4 * n * c["Hq"] * d}
    new = _spread(T, B, c["ragged"])
    pairs = sum(n * t + t * (t + 1) // (2 if not c["tree"] else 8) for n, t in zip(seen, new))
    return {"bytes": 2 * sum(seen) * H * held + 2 * sum(new) * H * d * e + 2 * sum(new) * c["Hq"] * d * e,
            "flops": 4 * pairs * c["Hq"] * d}


# ----------------------------------------------------------------- the definitions in 64 bits
def _exact_e4m3(x):
    """Rows in 64 bits to the values that their 8-bit form stands for."""
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-30) / 448)))
    y = x / scale
    _, e = torch.frexp(y)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step * scale


def _exact_rows(s):
    """The rows to be written, [B, H, N, d]."""
    c = s["case"]
    k, v = s["k"].double(), s["v"].double()
    if c["op"] == "store":
        h = c["d"] // 2
        ang = torch.stack([s["pos"][0].double() * f for f in s["inv_freq"].tolist()], -1)[:, None]
        z = torch.complex(k[..., :h], k[..., h:]) * torch.polar(torch.ones_like(ang), ang)
        k = torch.cat([z.real, z.imag], -1)
    else:
        pick = lambda x: torch.stack([x[b][:, s["path"][b].long()] for b in range(c["B"])])  # noqa: E731
        k, v = pick(k), pick(v)
    return (_exact_e4m3(k), _exact_e4m3(v)) if c["bits8"] else (k, v)


def _exact_write(s):
    """For every slot of every sequence the newest row that lands in it; then what is returned."""
    c = s["case"]
    ring = c["capacity"] - c["sinks"]
    rows = _exact_rows(s)
    out = tuple(torch.zeros_like(x) if c["bits8"] else s[n].double() for x, n in zip(rows, ("k_cache", "v_cache")))
    for b, (a, n) in enumerate(zip(s["lens"].tolist(), s["n_new"].tolist())):
        holds = {}
        for p in range(a, a + n):
            holds[p if p < c["sinks"] else c["sinks"] + (p - c["sinks"]) % ring] = p - a
        slot, t = torch.tensor(list(holds)), torch.tensor(list(holds.values()))
        to = t if c["bits8"] else slot                        # 8-bit caches are read back by position
        for y, x in zip(out, rows):
            y[b][:, to] = x[b][:, t]
    return out


def _exact_positions(s, b, L):
    """Positions that sequence b's cache holds, and their keys and values [Hkv, n, d] in 64 bits."""
    c = s["case"]
    ring = c["capacity"] - c["sinks"]
    p = torch.arange(L, device="cuda")
    p = p[(p < c["sinks"]) | (p >= L - ring)]
    slot = torch.where(p < c["sinks"], p, c["sinks"] + (p - c["sinks"]) % ring)

    def rows(x, scale):
        if scale is None:
            return x[b][:, slot].double()
        return x[b].double()[:, slot] * scale[b][:, slot, None].double()

    return p, rows(s["k_cache"], s["k_scale"]), rows(s["v_cache"], s["v_scale"])


def _exact_attention(s):
    c = s["case"]
    G, T = c["Hq"] // c["Hkv"], c["T"]
    o = torch.zeros((c["B"], c["Hq"], T, c["d"]), dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(zip(s["lens"].tolist(), s["n_new"].tolist())):
        p, k, v = _exact_positions(s, b, L)
        if c["op"] == "decode":
            at = torch.tensor([L - 1], device="cuda")
        else:
            parents = list(range(-1, T - 1)) if s["parents"] is None else s["parents"][b].tolist()
            line = []                                         # every node's ancestors and itself
            for t in range(n):
                line.append((line[parents[t]] if parents[t] >= 0 else []) + [t])
            at = torch.tensor([L + len(x) - 1 for x in line], device="cuda")
            of = torch.zeros((n, n), dtype=torch.bool)
            for t, x in enumerate(line):
                of[t, x] = True
            p, k, v = torch.cat([p, at]), torch.cat([k, s["k"][b, :, :n].double()], 1), torch.cat(
                [v, s["v"][b, :, :n].double()], 1)
        see = (p[None] <= at[:, None]) & ((p[None] > at[:, None] - c["window"]) | (p[None] < c["sinks"]))
        if c["op"] == "tree":
            see[:, -n:] &= of.cuda()
        for h in range(c["Hq"]):
            x = torch.einsum("id,jd->ij", s["q"][b, h, :n].double(), k[h // G]) * s["scale"]
            o[b, h, :n] = torch.softmax(x.masked_fill_(~see, -math.inf), -1) @ v[h // G]
    return o[:, :, 0] if c["op"] == "decode" else o


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_write(s) if case["op"] in ("store", "accept") else _exact_attention(s)
