"""8-bit rolling caches where they can go wrong: values of every size next to one another,
scales of every number, large queries, keys whose rotated maximum lies beside a border between two
scales, caches in every memory order, and what a call leaves behind.  On the GPU against the
oracle within the bounds that it derives."""
import gc
import math

import numpy as np
import pytest

import tree_oracle as T
import window_oracle as W
from self_attention_backward_gb300 import binding as B
from self_attention_backward_gb300.inputs import round_storage
from test_tree import ALGOS, DECODES, KINDS, Cache8, Tree, _close, _codes, _i32, _name, _visible_slots
from test_window import _dev, _draw, _gpu, _np, _plan, lib  # noqa: F401

ALGOS8 = [a for a in ALGOS if a[0][1]]


def _decode(cache, q, lens, scale, dtype, lse=None):
    return cache.decode(_dev(q, dtype, "bhnd")[:, :, 0], _i32(lens), scale, lse=lse)[:, :, None]


# ---------------------------------------------------------------- values of every size
def _sized_values(c, kind, up):
    """The values of a Cache8 or a Tree: rows of zeros as the cache's writes leave them (codes 0, scale
    2^-100) among rows 2^up times as large as before, in an order of positions."""
    torch = _gpu()
    cap = c.vals[1].shape[2]
    at = np.arange(cap)
    zero = {"first": at < cap // 2, "last": at >= cap // 2, "between": at % 3 == 1, "one large": at != cap // 2}[kind]
    s = c.vs if isinstance(c, Tree) else c.scales[1]
    code = c.vals[1] / s[..., None]
    code[:, :, zero], s[:, :, zero] = 0.0, 2.0 ** -100
    s[:, :, ~zero] *= 2.0 ** up
    c.vals[1][:] = code * s[..., None]
    raw = torch.from_numpy(code).to(torch.float32).to(torch.float8_e4m3fn)
    c.cache.v.view(torch.uint8).copy_(raw.view(torch.uint8))
    c.cache.v_scale.copy_(torch.from_numpy(s).float())


def _lost(c, n_kv):
    """What weights that are too small for fp32 may take from an output [B, Hq, T, d]: a key whose weight is
    below 2^-126 of the reference that its exponential is taken against (at most 2^8 below the row's
    largest) counts as 0, and so does what a row had before its reference moves by more than 2^126.  So
    each key loses at most 2^-118 of the row's largest weight, which is at most the row's sum: in all 2^-118
    times the sum of |v|."""
    return 2.0 ** -118 * np.repeat(np.abs(c.vals[1]).sum(2), n_kv, axis=1)[:, :, None]


SIZED = [(200, 190, [196]), (200, 190, [64]), (1000, 900, [950]), (2500, 2400, [2450])]   # one run of keys, a cluster's, more


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZED, ids=lambda s: f"{s[0]}-{s[2][0]}")
@pytest.mark.parametrize("up", [28, 64, 100])
@pytest.mark.parametrize("kind", ["first", "last", "between", "one large"])
def test_decode_zero_values_beside_large_ones(lib, dtype, size, up, kind):
    """A key counts in a row's sum whatever the size of its value."""
    torch = _gpu()
    cap, window, lens = size
    rng = np.random.default_rng(cap + up)
    d, scale = 64, 0.125
    c = Cache8(rng, 1, 2, cap, d, window, 4)
    _sized_values(c, kind, up)
    for heads in (8, 24):                                     # 4 and 12 rows of a key head
        q = _draw(rng, (1, heads, 1, d), dtype)
        lse = torch.empty((1, heads), device="cuda")
        o = _decode(c.cache, q, lens, scale, dtype, lse)
        ref = T.tree(q.astype(np.float64), *c.vals, None, None, lens, None, None, cap, window, 4, scale, W.U[dtype], c.scales[1])
        _close(o, ref[0], ref[2] + _lost(c, heads // 2), "O")
        _close(lse[..., None], ref[1], ref[3], "LSE")


@pytest.mark.gpu
@pytest.mark.parametrize("algo", ALGOS8, ids=_name)
@pytest.mark.parametrize("shape", [(4, 2, 3), (4, 2, 8), (4, 2, 14), (4, 1, 40)], ids=str)    # 6, 16, 28 and 160 rows
@pytest.mark.parametrize("up", [28, 100])
@pytest.mark.parametrize("kind", ["first", "last", "between", "one large"])
def test_tree_zero_values_beside_large_ones(lib, algo, shape, up, kind):
    """The same for drafted tokens, whose own values are of ordinary size."""
    torch = _gpu()
    Hq, Hkv, n = shape
    for cap, window, lens in SIZED:
        c = Tree(*algo[0], 64, 1, Hq, Hkv, n, cap, window, 4, lens, None, "tree", seed=up, garbage=False)
        _sized_values(c, kind, up)
        lse = torch.empty(c.x[0].shape[:3], device="cuda")
        o = c.run(algo[1], lse=lse)
        ref = T.tree(c.x[0], *c.vals, c.x[1], c.x[2], lens, c.real, c.parents, cap, window, 4, c.scale, W.U[c.dtype], c.vs)
        _close(o, ref[0], ref[2] + _lost(c, Hq // Hkv), "O")
        _close(lse, ref[1], ref[3], "LSE")


# ---------------------------------------------------------------- scales of every number
ANY_SCALE = [
    (3, 4, 2, 7, 300, 260, 3, [290, 100, 1000], [7, 5, 7], "tree"),
    (2, 32, 1, 9, 400, 390, 2, [390, 777], None, "chain"),
    (2, 8, 2, 40, 700, 600, 4, [650, 333], [40, 11], "tree"),
    (1, 4, 1, 130, 500, 480, 0, [485], None, "run"),
    (40, 2, 1, 20, 300, 260, 3, [0, 5, 130, 263, 999] * 8, None, "wild"),
]


def _as_documented(c, algo):
    """The cache's values as the kernel takes them: on the tensor cores code times scale, an fp32 product, is
    rounded to bf16; elsewhere the scale stays apart."""
    if algo == B.PSA_ALGO_TC:
        c.vals = [round_storage(x.astype(np.float32), "bf16").astype(np.float64) for x in c.vals]


def _any_scales(c, seed):
    """Scales as max / 448 makes them: any fp32 numbers."""
    torch = _gpu()
    rng = np.random.default_rng(seed)
    for i, to in enumerate((c.cache.k_scale, c.cache.v_scale)):
        s = to.double().cpu().numpy()
        new = (s * rng.uniform(1.0, 2.0, size=s.shape)).astype(np.float32).astype(np.float64)
        c.vals[i] *= (new / s)[..., None]
        to.copy_(torch.from_numpy(new).float())
        if i:
            c.vs = new


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("algo", ALGOS8, ids=_name)
@pytest.mark.parametrize("size", ANY_SCALE, ids=lambda s: "-".join(str(x) for x in s[:7]))
def test_tree_scales_of_any_number(lib, size, algo, d):
    """No rounding of cached elements but the tensor cores' documented one: with keys rounded to bf16 on the
    way most row sums would be off by several times their bounds."""
    _gpu()
    c = Tree(*algo[0], d, *size, seed=d, std=3.0, garbage=False)
    _any_scales(c, d)
    _as_documented(c, algo[1])
    c.check(algo[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads", [8, 24])
def test_decode_scales_of_any_number(lib, dtype, heads):
    """Single tokens have no such rounding."""
    torch = _gpu()
    c = Tree(dtype, True, 64, 2, heads, 2, 1, 400, 380, 4, [382, 1000], None, "run", seed=heads, std=3.0, garbage=False)
    _any_scales(c, heads)
    q, lse = c.x[0], torch.empty((2, heads), device="cuda")
    o = _decode(c.cache, q, c.lens, c.scale, dtype, lse)
    ref = T.tree(q, *c.vals, None, None, c.lens, None, None, *c.size, c.scale, W.U[dtype], c.vs)
    _close(o, ref[0], ref[2], "O")
    _close(lse[..., None], ref[1], ref[3], "LSE")


@pytest.mark.gpu
@pytest.mark.parametrize("algo", ALGOS8, ids=_name)
def test_tree_some_scales_of_any_number(lib, algo):
    """One such key, or one such value, in a tile of others; NaN in hidden places."""
    torch = _gpu()
    for at, which in ((3, 0), (131, 0), (270, 1), (200, 1)):
        c = Tree(*algo[0], 64, 2, 8, 2, 24, 400, 380, 4, [382, 383], None, "tree", seed=at)
        t = (c.cache.k_scale, c.cache.v_scale)[which]
        old = t[:, :, at].double().cpu().numpy()
        t[:, :, at] *= 1.3
        c.vals[which][:, :, at] *= (t[:, :, at].double().cpu().numpy() / old)[..., None]
        c.vs = c.cache.v_scale.double().cpu().numpy()
        c.vs[~np.isfinite(c.vs)] = 1.0
        _as_documented(c, algo[1])
        c.check(algo[1])


def test_bounds_see_keys_rounded_to_bf16():
    """The oracle with such keys is out of its own bounds, so the tests above would notice."""
    rng = np.random.default_rng(1)
    for d in (16, 64, 128):
        k = 3 * rng.normal(size=(1, 1, 300, d))
        q, v = round_storage(3 * rng.normal(size=(1, 8, 1, d)), "bf16").astype(np.float64), rng.normal(size=k.shape)
        args = (None, None, [296], None, None, 300, 290, 4, d ** -0.5, W.U["bf16"])
        o, lse, bo, bl = T.tree(q, k, v, *args)
        off = T.tree(q, round_storage(k, "bf16").astype(np.float64), v, *args)
        assert (np.abs(off[1] - lse) > 2 * bl).sum() >= 6


# ---------------------------------------------------------------- large queries and keys
@pytest.mark.gpu
@pytest.mark.parametrize("algo", ALGOS8, ids=_name)
@pytest.mark.parametrize("n", [2, 12])
def test_scores_of_zero_from_large_factors(lib, algo, n):
    """Queries of 2^100 in one feature, keys of 2^50 in the others: every score is 0."""
    torch = _gpu()
    c = Tree(*algo[0], 64, 1, 4, 1, n, 300, 290, 4, [280], None, "tree", seed=n, garbage=False)
    q, kn, vn = c.x
    q[..., 0], q[..., 1:], kn[..., 0] = 2.0 ** 100, 0.0, 0.0
    c.cache.k.view(torch.uint8)[..., 0] = 0
    c.cache.k_scale.mul_(2.0 ** 50)
    c.t = [_dev(x, c.dtype) for x in c.x]
    ref = T.tree(0 * q, 0 * c.vals[0], c.vals[1], 0 * kn, vn, c.lens, c.real, c.parents, *c.size, c.scale, W.U[c.dtype], c.vs)
    lse = torch.empty(q.shape[:3], device="cuda")
    o = c.run(algo[1], lse=lse)
    _close(o, ref[0], ref[2], "O")
    _close(lse, ref[1], ref[3], "LSE")
    at = (c.lens, None, None, *c.size, c.scale, W.U[c.dtype], c.vs)
    ref = T.tree(0 * q[:, :, :1], 0 * c.vals[0], c.vals[1], None, None, *at)
    _close(_decode(c.cache, q[:, :, :1], c.lens, c.scale, c.dtype), ref[0], ref[2], "decode")


# ---------------------------------------------------------------- scales of rotated keys
def _border_keys(rng, dtype, want):
    """Pairs (x1, x2) and positions whose first rotated feature is the pair's larger one, and within
    2^-25 .. 2^-23 of 448 2^-8 (1.75) on either side: nearer than an fp32 rotation is sure of, farther
    than the 2^-26 of it that cosines and sines off by 2^-27 make."""
    found = []
    while sum(len(x[0]) for x in found) < want:
        n = 1 << 20
        x1 = round_storage(rng.uniform(-2.0, 2.0, size=n), dtype).astype(np.float64)
        pos = rng.integers(1, 100000, size=n)
        c, s = np.cos(pos.astype(np.float64)), np.sin(pos.astype(np.float64))
        with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
            x2 = (x1 * c - 1.75 * (1 + rng.choice([-1, 1], size=n) * 2.0 ** rng.uniform(-25, -23, size=n))) / s
        x2 = round_storage(np.where(np.abs(x2) < 4, x2, 0.0), dtype).astype(np.float64)
        y1, y2 = x1 * c - x2 * s, x2 * c + x1 * s
        d = np.abs(y1 / 1.75 - 1)
        hit = (d > 2.0 ** -25) & (d < 2.0 ** -23) & (np.abs(y2) < 0.9 * np.abs(y1))
        found.append([z[hit] for z in (x1, x2, pos, y1, y2)])
    return [np.concatenate([f[i] for f in found])[:want] for i in range(5)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("layout", ["bnhd", "odd"])
def test_store_8bit_scale_of_the_exact_rotation(lib, dtype, inter, layout):
    """The scale is that of the exactly rotated key's maximum, and the codes are x over that scale."""
    torch = _gpu()
    rng = np.random.default_rng(3)
    n, d = 240, 64
    x1, x2, pos, y1, y2 = _border_keys(rng, dtype, n)
    plan = _plan(head_dim=d, sections=(8,), rot_dim=16, interleaved=inter)
    k = np.zeros((1, 1, n, d))
    k[..., 16:] = round_storage(rng.normal(size=(1, 1, n, d - 16)) * 2.0 ** rng.integers(-13, -1, size=(1, 1, n, d - 16)), dtype)
    k[..., 16:] = np.clip(k[..., 16:], -1.0, 1.0)
    exact = k.copy()
    f1, f2 = (0, 1) if inter else (0, 8)
    k[0, 0, :, f1], k[0, 0, :, f2], exact[0, 0, :, f1], exact[0, 0, :, f2] = x1, x2, y1, y2
    up = 2.0 ** rng.integers(-30, 31, size=(1, 1, n, 1))     # the same at other exponents
    k, exact = k * up, exact * up
    c = Cache8(rng, 1, 1, n, d, n - 4, 4)
    t = _dev(k, dtype, layout)
    c.cache.append(t, t.clone(), _i32([0]), plan=plan, pos=_i32(pos[None, None].tolist()))
    s = np.where(np.abs(y1) > 1.75, 2.0 ** -7, 2.0 ** -8)[None, None, :, None] * up
    assert np.array_equal(c.ks.double().cpu().numpy(), s[..., 0])
    y = exact / s
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 1e-30))), -6) - 3)
    tie = np.abs(np.abs(y / step - np.floor(y / step)) - 0.5) < 2.0 ** -20
    tie[..., 16:] = False                                     # copied features are exact: ties go to even
    assert tie.mean() < 1e-3 and ((_codes(c.cache.k) == np.rint(y / step) * step) | tie).all()


# ---------------------------------------------------------------- memory orders
@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["bnhd", "odd"])
@pytest.mark.parametrize("size", DECODES[3:10], ids=lambda s: "-".join(str(x) for x in s[:6]))
def test_decode_8bit_memory_orders(lib, size, layout, dtype, d):
    """Token-major caches and rows of d + 3 codes: what the head-major cache gives."""
    torch = _gpu()
    Bn, Hq, Hkv, cap, window, sinks, lens = size
    got = []
    for at in ("bhnd", layout):
        rng = np.random.default_rng(cap + Hq)
        c = Cache8(rng, Bn, Hkv, cap, d, window, sinks, at)
        c.hide(lambda b: _visible_slots(lens[b], cap, window, sinks))
        q = _draw(rng, (Bn, Hq, 1, d), dtype)
        got.append(_decode(c.cache, q, lens, 1 / math.sqrt(d), dtype))
    assert torch.isfinite(got[0]).all() and torch.equal(*got)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("algo", ALGOS8, ids=_name)
@pytest.mark.parametrize("layout", ["bnhd", "odd"])
@pytest.mark.parametrize("n", [1, 2, 30])
def test_tree_8bit_memory_orders(lib, algo, layout, d, n):
    """1, 2 and 30 tokens of 4 heads a key head; odd rows are not the tensor cores' to take."""
    torch = _gpu()
    c = Tree(*algo[0], d, 3, 8, 2, n, 300, 260, 3, [290, 100, 1000], None, "tree", seed=d)
    want = c.check(algo[1])
    t = [c.cache.k.view(torch.uint8), c.cache.v.view(torch.uint8), c.cache.k_scale, c.cache.v_scale]
    if layout == "bnhd":
        t = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in t]
    else:
        wide = [torch.full((*x.shape[:3], d + 3), 0x7F, dtype=torch.uint8, device="cuda") for x in t[:2]]
        for w, x in zip(wide, t):
            w[..., :d] = x
        t = [w[..., :d] for w in wide] + [x.transpose(1, 2).contiguous().transpose(1, 2) for x in t[2:]]
    f8 = torch.float8_e4m3fn
    c.cache = B.WinCache(t[0].view(f8), t[1].view(f8), 260, 3, t[2], t[3])
    if layout == "odd" and algo[1] == B.PSA_ALGO_TC:
        with pytest.raises(B.PsaError) as e:
            c.run(algo[1])
        assert e.value.code == B.PSA_ERR_UNSUPPORTED
    else:
        assert torch.equal(c.run(algo[1]), want)


# ---------------------------------------------------------------- calls
def test_append_takes_its_stream_seventh(lib, monkeypatch):
    """append(k_new, v_new, start, n_new, plan, pos, stream): the order before there were rows."""
    torch = pytest.importorskip("torch")
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    c = B.WinCache(z(1, 2, 8, 32), z(1, 2, 8, 32), 4, 1)
    seen = []
    monkeypatch.setattr(B, "_on_stream", lambda stream, device, f, *a, **kw: seen.append((stream, a, kw)))
    c.append(z(1, 2, 3, 32), z(1, 2, 3, 32), z(1, t=torch.int32), None, None, None, 1234)
    assert len(seen) == 1 and seen[0][0] == 1234


@pytest.mark.gpu
def test_append_by_index_on_a_stream(lib):
    """rows and a stream together."""
    torch = _gpu()
    rng = np.random.default_rng(2)
    k, v = (_dev(_draw(rng, (1, 2, 6, 32), "bf16"), "bf16", "bhnd") for _ in range(2))
    c = B.WinCache(*(torch.zeros((1, 2, 8, 32), dtype=torch.bfloat16, device="cuda") for _ in range(2)), 4, 1)
    start, rows = _i32([2]), _i32([[5, 0, 3]])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    c.append(k, v, start, None, None, None, s, rows)
    s.synchronize()
    assert torch.equal(c.k[:, :, 2:5], k[:, :, [5, 0, 3]]) and torch.equal(c.v[:, :, 2:5], v[:, :, [5, 0, 3]])


# ---------------------------------------------------------------- workspaces
@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS, ids=_name)
def test_calls_keep_no_memory(lib, kind):
    """Many caches (a model has one a layer): what a call works in is given back."""
    torch = _gpu()
    cases = [Tree(*kind, 128, 2, 8, 2, 100, 2100, 2048, 4, [2000, 5000], None, "tree", seed=s, garbage=False) for s in range(4)]
    lens, par = _i32(cases[0].lens), _i32(cases[0].parents.tolist())
    c = cases[0]
    c.cache.tree(*c.t, lens, c.scale, parents=par)            # loads the kernels
    torch.cuda.synchronize()
    gc.collect()                                              # what earlier tests left is not to be given back meanwhile
    before = torch.cuda.memory_allocated()
    for c in cases:
        for n in (100, 40, 3):
            c.cache.tree(*(x[:, :, :n] for x in c.t), lens, c.scale, parents=par[:, :n].contiguous())
        if kind[1]:
            c.cache.decode(c.t[0][:, :, 0], lens, c.scale)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS, ids=_name)
def test_two_graphs_of_one_cache_at_once(lib, kind):
    """Two captured calls over one cache, replayed side by side on two streams."""
    torch = _gpu()
    c = Tree(*kind, 128, 2, 8, 2, 40, 2100, 2048, 4, [2000, 5000], None, "tree", seed=1, garbage=False)
    lens, par = _i32(c.lens), [_i32(c.parents.tolist()), None]
    run = lambda i: c.cache.tree(*c.t, lens, c.scale, parents=par[i])  # noqa: E731
    want = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            got.append(run(i))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(w, x) for w, x in zip(want, got))


# ---------------------------------------------------------------- which kernel
@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    # sequences of 8 key heads, 4 query heads each, tokens, window, whether the tensor cores are faster
    (19, 4, 1024, True), (16, 4, 4096, False), (1, 4, 4096, True), (1, 4, 512, False), (16, 8, 4096, True), (1, 2, 1024, False),
], ids=str)
def test_auto_takes_the_faster_kernel_over_8bit_caches(lib, case):
    """What the rule's measured sizes say, seen by the bits: the kernels round differently."""
    torch = _gpu()
    Bn, n, window, tensor_cores = case
    g = torch.Generator(device="cuda").manual_seed(1)
    shape = (Bn, 8, window + 4, 128)
    code = [torch.randint(0, 100, shape, generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in "kv"]
    c = B.WinCache(*code, window, 4, *(torch.full(shape[:3], 2.0 ** -4, device="cuda") for _ in "kv"))
    q, k, v = (torch.randn((Bn, h, n, 128), generator=g, device="cuda").to(torch.bfloat16) for h in (32, 8, 8))
    lens = torch.full((Bn,), 2 * window, dtype=torch.int32, device="cuda")
    auto, warps, tc = (c.tree(q, k, v, lens, 0.088, algo=x) for x in (B.PSA_ALGO_AUTO, B.PSA_ALGO_SIMT, B.PSA_ALGO_TC))
    assert not torch.equal(warps, tc)
    assert torch.equal(auto, tc if tensor_cores else warps)
