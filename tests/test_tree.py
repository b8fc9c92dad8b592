"""The rolling cache in 8 bits (quantised as it is written, read back, single tokens over
it), accepted paths, and the attention of drafted tokens over caches of every type: refusals
and the oracle's own checks on the CPU; on the GPU, every operator against the oracle within
the bounds that it derives, and runs of them together."""
import math

import numpy as np
import pytest

import tree_oracle as T
import window_oracle as W
from self_attention_backward_gb300 import binding as B
from self_attention_backward_gb300.inputs import round_storage
from test_window import FAKE, INF, _cache, _dev, _draw, _gpu, _np, _plan, _view, lib  # noqa: F401


def _close(got, ref, bound, what):
    """Finite where the reference is and within the derived bound there, equal elsewhere."""
    got = _np(got)
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin]), what
    err = np.abs(got[fin] - ref[fin])
    over = ~(err <= bound[fin] + 1e-30)
    assert not over.any(), (what, float((err[over] / (bound[fin][over] + 1e-30)).max()), int(over.sum()))


# ---------------------------------------------------------------- the oracle itself
def test_oracle_run_is_the_windowed_attention():
    """A run of tokens over a cache that holds everything: the last rows of the forward."""
    rng = np.random.default_rng(1)
    L, n, d, window, sinks = 20, 6, 8, 7, 2
    q, k, v = (rng.normal(size=(L + n, d)) for _ in range(3))
    want = W.attention(q[L:], k, v, 0.4, window, sinks)
    got = T.tree(q[None, None, L:], k[None, None, :L], v[None, None, :L], k[None, None, L:], v[None, None, L:], [L], [n], None,
                 L + 5, window, sinks, 0.4, 0.0)
    np.testing.assert_allclose(got[0][0, 0], want[0], rtol=1e-12)
    np.testing.assert_allclose(got[1][0, 0], want[1], rtol=1e-12)


def test_oracle_tree_node_is_its_path():
    """A node's output is that of its path, appended and asked for by its last token."""
    rng = np.random.default_rng(2)
    L, n, d, cap, window, sinks = 30, 7, 8, 16, 11, 2
    k, v = rng.normal(size=(2, cap, d))
    q, kn, vn = (rng.normal(size=(n, d)) for _ in range(3))
    parents = [-1, 0, 0, 1, 3, -1, 2]
    o = T.tree(q[None, None], k[None, None], v[None, None], kn[None, None], vn[None, None], [L], [n], [parents], cap, window,
               sinks, 0.5, 0.0)[0][0, 0]
    for t in range(n):
        path = np.nonzero(T.ancestors(parents, n)[t])[0]
        kc, vc = k.copy(), v.copy()
        for i, x in enumerate(path):
            s = W.slot(L + i, cap, sinks)
            kc[s], vc[s] = kn[x], vn[x]
        want = T.tree(q[None, None, t:t + 1], kc[None, None], vc[None, None], None, None, [L + len(path)], None, None, cap,
                      window, sinks, 0.5, 0.0)[0][0, 0, 0]
        np.testing.assert_allclose(o[t], want, rtol=1e-12)


def test_oracle_quantises_to_the_nearest_code():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(40, 16)).astype(np.float32).astype(np.float64) * 10.0 ** rng.integers(-20, 20, size=(40, 1))
    x[0], x[1, 3], x[2] = 0.0, np.nan, np.sign(x[2]) * 448 * 2.0 ** -7
    codes, s, _ = T.quantise(x)
    table = T.e4m3_table()
    table = table[np.isfinite(table)]
    assert np.isnan(s[1]) and s[0] == 2.0 ** -100 and s[2] == 2.0 ** -7
    for r in range(2, 40):
        assert np.abs(x[r]).max() <= 448 * s[r] and np.abs(x[r]).max() > 224 * s[r]
        near = np.abs(x[r][:, None] / s[r] - table[None]).min(-1)
        np.testing.assert_array_equal(np.abs(x[r] / s[r] - codes[r]), near)


# ---------------------------------------------------------------- refusals (nothing is launched)
def _cache8(**kw):
    return _cache(**dict(dict(dtype=B.PSA_E4M3), **kw))


def _scales(**kw):
    a = dict(k=FAKE, v=FAKE * 32, batch_stride=16, head_stride=8, slot_stride=1)
    a.update(kw)
    return B.psa_win_scales(*a.values())


def _calls(lib):
    """Every new entry point as f(cache, scales, **changes)."""
    v = _view()

    def store(c, s, k=v, T=8, rows=None, rs=0, R=8, start=FAKE, n=None, plan=None, pos=None, dt=B.PSA_BF16):
        return lib.psa_win_store(c, s, k, v, T, rows, rs, R, start, n, plan, pos, 0, 0, dt, None)

    def read(c, s, k=v, N=8, first=FAKE, lens=FAKE, dt=B.PSA_BF16):
        return lib.psa_win_read(c, s, k, v, N, first, lens, dt, None)

    def decode(c, s, q=v, o=v, lse=None, heads=4, lens=FAKE, scale=0.5, ws=FAKE, n=1 << 40, dt=B.PSA_BF16):
        return lib.psa_win_decode_any(c, s, q, o, lse, heads, lens, scale, ws, n, dt, None)

    def tree(c, s, q=v, kn=v, o=v, lse=None, heads=4, T=8, par=None, ps=0, nn=None, lens=FAKE, scale=0.5, ws=FAKE, n=1 << 40,
             algo=0, dt=B.PSA_BF16):
        return lib.psa_win_tree_attn(c, s, q, kn, v, o, lse, heads, T, par, ps, nn, lens, scale, ws, n, algo, dt, None)

    return store, read, decode, tree


@pytest.mark.parametrize("kw,code", [
    (dict(capacity=4), B.PSA_ERR_ARG), (dict(head_dim=8), B.PSA_ERR_UNSUPPORTED), (dict(dtype=3), B.PSA_ERR_ARG),
    (dict(v=FAKE + 8), B.PSA_ERR_ALIGN), (dict(slot_stride=0), B.PSA_ERR_ARG), (dict(window=0, capacity=1), B.PSA_ERR_ARG),
    (dict(sinks=-1), B.PSA_ERR_ARG),
])
def test_new_calls_refuse_caches(lib, kw, code):
    for call in _calls(lib):
        assert call(_cache8(**kw), _scales()) == code
        assert B.psa_attn_last_error()
    assert lib.psa_win_tree_attn_workspace_bytes(_cache8(**kw), 4, 8, B.PSA_BF16) == 0
    assert lib.psa_win_decode_any_workspace_bytes(_cache8(**kw), 4, B.PSA_BF16) == 0


def test_new_calls_refuse_scales_and_types(lib):
    for call in _calls(lib):
        assert call(_cache8(), None) == B.PSA_ERR_ARG
        assert call(_cache(), _scales()) == B.PSA_ERR_ARG
        assert call(_cache8(), _scales(k=None)) == B.PSA_ERR_ARG
        assert call(_cache8(), _scales(k=FAKE * 32)) == B.PSA_ERR_ARG
        assert call(_cache8(), _scales(v=FAKE + 2)) == B.PSA_ERR_ALIGN
        assert call(_cache8(), _scales(slot_stride=0)) == B.PSA_ERR_ARG
        assert call(_cache8(), _scales(head_stride=-1)) == B.PSA_ERR_ARG
        assert call(_cache8(), _scales(slot_stride=1 << 41)) == B.PSA_ERR_UNSUPPORTED
        assert call(_cache8(), _scales(), dt=B.PSA_E4M3) == B.PSA_ERR_ARG
    store, read, decode, tree = _calls(lib)
    for call in (store, decode, tree):
        assert call(_cache(), None, dt=B.PSA_F32) == B.PSA_ERR_ARG
    c = _cache8()
    v = _view()
    assert lib.psa_win_cache_append(c, v, v, 8, FAKE, None, None, None, 0, 0, None) == B.PSA_ERR_ARG
    assert lib.psa_win_decode(c, v, v, None, 4, FAKE, 0.5, FAKE, 1 << 40, None) == B.PSA_ERR_ARG


def test_new_calls_refuse_arguments(lib):
    store, read, decode, tree = _calls(lib)
    c, s, p = _cache8(), _scales(), _plan().c
    assert store(c, s, k=None) == B.PSA_ERR_ARG
    assert store(c, s, T=-1) == B.PSA_ERR_ARG
    assert store(c, s, R=7) == B.PSA_ERR_ARG                  # fewer positions than rows, and no rows named
    assert store(c, s, rows=FAKE, R=-1) == B.PSA_ERR_ARG
    assert store(c, s, rows=FAKE, rs=-1) == B.PSA_ERR_ARG
    assert store(c, s, rows=FAKE + 2) == B.PSA_ERR_ALIGN
    assert store(c, s, start=None) == B.PSA_ERR_ARG
    assert store(c, s, plan=p) == B.PSA_ERR_ARG
    assert store(c, s, T=0, R=0, k=None, start=None) == B.PSA_OK
    assert read(c, s, N=-1) == B.PSA_ERR_ARG
    assert read(c, s, first=None) == B.PSA_ERR_ARG
    assert read(c, s, lens=FAKE + 1) == B.PSA_ERR_ALIGN
    assert read(c, s, k=_view(sn=0)) == B.PSA_ERR_ARG
    assert read(c, s, N=0, k=None, first=None) == B.PSA_OK
    assert decode(c, s, heads=3) == B.PSA_ERR_ARG
    assert decode(c, s, lens=None) == B.PSA_ERR_ARG
    assert decode(c, s, scale=INF) == B.PSA_ERR_ARG
    assert decode(c, s, o=_view(sh=0)) == B.PSA_ERR_ARG
    assert decode(c, s, lse=FAKE + 2) == B.PSA_ERR_ALIGN
    assert tree(c, s, T=B.PSA_TREE_MAX + 1) == B.PSA_ERR_UNSUPPORTED
    assert tree(c, s, T=-1) == B.PSA_ERR_ARG
    assert tree(c, s, heads=3) == B.PSA_ERR_ARG
    assert tree(c, s, q=None) == B.PSA_ERR_ARG
    assert tree(c, s, kn=_view(0)) == B.PSA_ERR_ARG
    assert tree(c, s, o=_view(sn=0)) == B.PSA_ERR_ARG
    assert tree(c, s, lens=None) == B.PSA_ERR_ARG
    assert tree(c, s, par=FAKE + 2) == B.PSA_ERR_ALIGN
    assert tree(c, s, par=FAKE, ps=-1) == B.PSA_ERR_ARG
    assert tree(c, s, nn=FAKE + 1) == B.PSA_ERR_ALIGN
    assert tree(c, s, scale=float("nan")) == B.PSA_ERR_ARG
    assert tree(c, s, algo=3) == B.PSA_ERR_ARG
    assert tree(c, s, T=0, q=None, lens=None) == B.PSA_OK
    assert tree(_cache8(B=0), s, q=None) == B.PSA_OK
    big = _cache8(capacity=1 << 20, window=1 << 19, batch_stride=1 << 26, head_stride=1 << 25)
    sc = _scales(batch_stride=1 << 21, head_stride=1 << 20)
    need = lib.psa_win_tree_attn_workspace_bytes(big, 4, 8, B.PSA_BF16)
    assert need > 0
    assert tree(big, sc, n=need - 1) == B.PSA_ERR_WORKSPACE
    assert tree(big, sc, ws=None) == B.PSA_ERR_WORKSPACE
    assert tree(big, sc, ws=FAKE + 4) == B.PSA_ERR_ALIGN


def test_binding_refuses(lib):
    torch = pytest.importorskip("torch")
    f8 = torch.zeros((1, 2, 8, 32), dtype=torch.uint8).view(torch.float8_e4m3fn)
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    sc = z(1, 2, 8, t=torch.float32)
    c16, c8 = B.WinCache(z(1, 2, 8, 32), z(1, 2, 8, 32), 4, 1), B.WinCache(f8, f8.clone(), 4, 1, sc, sc.clone())
    q, kn, i = z(1, 4, 3, 32), z(1, 2, 3, 32), z(1, t=torch.int32)
    bad = [
        lambda: B.WinCache(f8, f8, 4, 1), lambda: B.WinCache(f8, f8, 4, 1, sc), lambda: B.WinCache(f8, f8, 4, 1, sc, sc[..., :4]),
        lambda: B.WinCache(f8, f8, 4, 1, sc, sc.double()), lambda: B.WinCache(z(1, 2, 8, 32), z(1, 2, 8, 32), 4, 1, sc, sc),
        lambda: c16.tree(q[0], kn, kn, i, 1.0), lambda: c16.tree(q, kn, kn, i, 1.0),           # the second: not on a GPU
        lambda: c8.read(i, 3, i), lambda: c8.read(i, -1, i), lambda: c8.read(i, 3, i, dtype=torch.float16),
        lambda: c8.append(kn, kn, i), lambda: c16.append(kn, kn, i, rows=z(3, t=torch.int64)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- GPU: writing and reading 8 bits
def _i32(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _codes(t):
    """float8 tensor -> its values."""
    return t.float().double().cpu().numpy()


class Cache8:
    """An 8-bit cache on the GPU whose slots hold random rows, and its values."""

    def __init__(self, rng, Bn, Hkv, cap, d, window, sinks, layout="bhnd", std=1.0, dtype="f32"):
        import torch
        self.vals, t, self.scales = [], [], []
        for _ in range(2):
            x = rng.normal(size=(Bn, Hkv, cap, d)) * std * np.exp(rng.normal(size=(Bn, Hkv, cap, 1)))
            code, s, f8 = T.quantise(x.astype(np.float32))
            self.vals.append(code * s[..., None])
            self.scales.append(s)
            raw = f8.view(torch.uint8).cuda()
            if layout == "bnhd":
                raw = raw.transpose(1, 2).contiguous().transpose(1, 2)
            elif layout == "odd":
                big = torch.full((Bn, Hkv, cap, d + 3), 0x7F, dtype=torch.uint8, device="cuda")
                big[..., :d] = raw
                raw = big[..., :d]
            ts = torch.from_numpy(s).float().cuda()
            if layout != "bhnd":
                ts = ts.transpose(1, 2).contiguous().transpose(1, 2)
            t += [raw, ts]
        self.k8, self.ks, self.v8, self.vs = t
        self.cache = B.WinCache(self.k8.view(torch.float8_e4m3fn), self.v8.view(torch.float8_e4m3fn), window, sinks, self.ks,
                                self.vs)

    def hide(self, slots_of):
        """NaN in every slot that slots_of(b) does not name."""
        for b in range(self.k8.shape[0]):
            seen = slots_of(b)
            hidden = [s for s in range(self.k8.shape[2]) if s not in seen]
            if hidden:
                for raw, s in ((self.k8, self.ks), (self.v8, self.vs)):
                    raw[b, :, hidden] = 0x7F
                    s[b, :, hidden] = float("nan")


STORES = [(1, 9, 2, [0, 1, 500], None), (5, 9, 2, [0, 7, 3], [5, 0, 2]), (40, 9, 2, [0, 7, 1], None),
          (40, 9, 0, [3, 9, 2], [40, 1, 77]), (6, 10, 3, [-1, 2 ** 31 - 4, 1], None), (700, 300, 4, [0, 31, 2], None)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["bnhd", "odd", "chan"])
@pytest.mark.parametrize("store", STORES, ids=lambda s: f"{s[0]}-{s[1]}-{s[2]}")
def test_store_8bit(lib, dtype, layout, store):
    """Codes and scales bit for bit by the definition; other slots hold what they held."""
    torch = _gpu()
    n, cap, sinks, start, n_new = store
    rng = np.random.default_rng(n + cap)
    Bn, Hkv, d = 3, 2, 32
    c = Cache8(rng, Bn, Hkv, cap, d, max(1, cap - sinks - 2), sinks, "odd" if layout == "odd" else "bhnd")
    kn, vn = (_draw(rng, (Bn, Hkv, n, d), dtype) * 4.0 ** rng.integers(-6, 7, size=(Bn, Hkv, n, 1)) for _ in range(2))
    want = [[_codes(t.view(torch.float8_e4m3fn)), _np(s)] for t, s in ((c.k8, c.ks), (c.v8, c.vs))]
    c.cache.append(_dev(kn, dtype, layout), _dev(vn, dtype, layout), _i32(start), None if n_new is None else _i32(n_new))
    for w, x in zip(want, (kn, vn)):
        code, s, _ = T.quantise(x)
        for b in range(Bn):
            m = n if n_new is None else min(max(n_new[b], 0), n)
            if start[b] < 0 or start[b] + m > 2 ** 31:
                continue
            for t in range(m):
                at = W.slot(start[b] + t, cap, sinks)
                w[0][b, :, at], w[1][b, :, at] = code[b, :, t], s[b, :, t]
    for w, t, s in zip(want, (c.k8, c.v8), (c.ks, c.vs)):
        assert np.array_equal(_codes(t.view(torch.float8_e4m3fn)), w[0]) and np.array_equal(_np(s), w[1])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_store_8bit_ends_of_the_range(lib, dtype, d):
    """Zeros, the smallest and largest numbers, ties, maxima at the scales' borders, and rows with
    an element that is not finite."""
    torch = _gpu()
    rng = np.random.default_rng(d)
    x = np.zeros((1, 1, 14, d), dtype=np.float64)
    x[0, 0, 1, 0] = 2.0 ** -126
    x[0, 0, 2] = 3e-38 * rng.normal(size=d)
    x[0, 0, 3] = 3e38 * rng.uniform(-1, 1, size=d)
    x[0, 0, 4, :4] = [448, 1.0625, 1.1875, 2.0 ** -10]        # ties between two codes
    x[0, 0, 5, :2] = [449, -3.0]
    x[0, 0, 6, :2] = [450, 2.0 ** -9 * 1.5]
    x[0, 0, 7, -1] = 448 * 2.0 ** 30
    x[0, 0, 8, -1] = -452 * 2.0 ** -30
    x[0, 0, 9] = rng.normal(size=d)
    x[0, 0, 10] = rng.normal(size=d)
    x[0, 0, 11] = 448 * 2.0 ** -100
    x[0, 0, 12] = 2.0 ** -103 * rng.normal(size=d)
    x[0, 0, 13] = np.float64(np.finfo(np.float32).max) if dtype == "f32" else 2.0 ** 127
    x = round_storage(x, dtype)
    x[0, 0, 9, 3], x[0, 0, 10, d - 1] = np.nan, -np.inf
    c = Cache8(rng, 1, 1, 20, d, 15, 2)
    t = _dev(x, dtype)
    c.cache.append(t, t.clone(), _i32([0]))
    code, s, _ = T.quantise(x)
    for raw, sc in ((c.k8, c.ks), (c.v8, c.vs)):
        assert np.array_equal(_codes(raw.view(torch.float8_e4m3fn))[:, :, :14], code)
        assert np.array_equal(_np(sc)[:, :, :14], s, equal_nan=True)
    k, v = c.cache.read(_i32([0]), 14, _i32([14]), dtype=torch.float32)
    with np.errstate(over="ignore"):                          # 256 * 2^120 is past the largest fp32 number
        want = (code * s[..., None]).astype(np.float32)
    assert np.array_equal(_np(k), want, equal_nan=True) and np.array_equal(_np(v), want, equal_nan=True)


ROTS = [((32,), None, False, 64), ((8, 12, 12), None, False, 64), ((4,), 8, False, 32), ((5,), 10, False, 64),
        ((16, 24, 24), None, True, 128), ((3,), 6, True, 16), ((8,), 16, False, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["bnhd", "odd"])
@pytest.mark.parametrize("rot", ROTS, ids=str)
def test_store_8bit_rotates(lib, dtype, layout, rot):
    """Read back in fp32: within half a code's step (2^-4 of it, or 2^-10 scales below the normal
    ones) of the rotated key, whose own error is the angle's (2^-26 turns, the sine's 2^-22) and
    three fp32 operations on |x1| + |x2|."""
    torch = _gpu()
    sections, rd, inter, d = rot
    rng = np.random.default_rng(d)
    Bn, Hkv, n, cap = 2, 3, 50, 64
    plan = _plan(head_dim=d, sections=sections, rot_dim=rd, interleaved=inter)
    c = Cache8(rng, Bn, Hkv, cap, d, 60, 4)
    kn, vn = _draw(rng, (Bn, Hkv, n, d), dtype), _draw(rng, (Bn, Hkv, n, d), dtype)
    pos = rng.integers(0, 99999, size=(len(sections), Bn, n)).astype(np.int32)
    c.cache.append(_dev(kn, dtype, layout), _dev(vn, dtype, layout), _i32([0, 5]), plan=plan, pos=torch.from_numpy(pos).cuda())
    k, v = c.cache.read(_i32([0, 5]), n, _i32([n, n + 5]), dtype=torch.float32)
    ref, mag = W.rotation(kn, pos, sections, 10000.0, False, inter, False)
    err = mag * (2 * math.pi * 2.0 ** -26 + 2.0 ** -22 + 3 * W.U32)
    top = np.abs(ref).max(-1, keepdims=True) + err.max(-1, keepdims=True)
    scale = 2.0 ** np.ceil(np.log2(top / 448))
    _close(k, ref, (np.abs(ref) + err) * 2.0 ** -4 + 2.0 ** -10 * scale + err, "rotated keys")
    code, s, _ = T.quantise(vn)
    assert np.array_equal(_np(v), code * s[..., None])


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("layout", ["bnhd", "odd"])
def test_store_8bit_codes_of_the_exact_rotation(lib, layout, inter):
    """Every code is the nearest one of the rotated key, unless that lies within 2^-26 (|x1| + |x2|)
    of the middle between two: cosine and sine are off by 2^-27 at most."""
    torch = _gpu()
    rng = np.random.default_rng(41)
    Bn, Hkv, n, d = 2, 4, 150, 128
    plan = _plan(head_dim=d, sections=(64,), rot_dim=d, interleaved=inter)
    c = Cache8(rng, Bn, Hkv, 200, d, 190, 4)
    kn, vn = _draw(rng, (Bn, Hkv, n, d), "bf16"), _draw(rng, (Bn, Hkv, n, d), "bf16")
    pos = rng.integers(0, 99999, size=(1, Bn, n)).astype(np.int32)
    c.cache.append(_dev(kn, "bf16", layout), _dev(vn, "bf16", layout), _i32([0, 0]), plan=plan, pos=torch.from_numpy(pos).cuda())
    ref, mag = W.rotation(kn, pos, (64,), 10000.0, False, inter, False)
    s = c.ks.double().cpu().numpy()[:, :, :n, None]
    top = np.abs(ref).max(-1, keepdims=True)
    assert (top <= 448 * s * (1 + 2.0 ** -24)).all() and (top > 224 * s * (1 - 2.0 ** -24)).all()
    y = ref / s
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 1e-30))), -6) - 3)
    tie = np.abs(y / step - np.floor(y / step) - 0.5) * step * s < mag * 2.0 ** -26
    want = np.rint(y / step) * step
    got = _codes(c.cache.k)[:, :, :n]
    assert tie.mean() < 1e-4 and ((got == want) | tie).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["f32", "bf16", "8 f32", "8 bf16"])
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("layout", ["bnhd", "odd"])
def test_append_of_an_accepted_path(lib, kind, rotated, layout):
    """The named rows, as if they had been gathered first: the same bits; a row out of range
    leaves its position, repeated rows and rows shared by the batch are fine."""
    torch = _gpu()
    rng = np.random.default_rng(21)
    dtype, Bn, Hkv, n, d, cap, sinks = kind[-4:].strip(), 3, 2, 30, 64, 12, 2
    kn, vn = (_dev(_draw(rng, (Bn, Hkv, n, d), dtype), dtype, layout) for _ in range(2))
    pos = torch.randint(0, 9999, (1, Bn, n), dtype=torch.int32, device="cuda") if rotated else None
    plan = _plan(head_dim=d, sections=(32,)) if rotated else None

    def make():
        r = np.random.default_rng(5)
        if kind[0] == "8":
            c = Cache8(r, Bn, Hkv, cap, d, 9, sinks)
            return c.cache, [c.k8, c.v8, c.ks, c.vs]
        t = [_dev(_draw(r, (Bn, Hkv, cap, d), dtype), dtype, "bhnd") for _ in range(2)]
        return B.WinCache(*t, 9, sinks), t

    for rows, n_new, start in (([[0, 3, 7, 29], [5, 5, 2, 1], [28, 0, 9, 4]], [4, 2, 3], [0, 7, 2 ** 31 - 5]),
                               ([[4, 1, 0]], None, [1, 1, 30]), ([list(range(25)) for _ in range(3)], [25, 25, 20], [3, 1, 0])):
        tr = _i32(rows)
        got, a = make()
        got.append(kn, vn, _i32(start), None if n_new is None else _i32(n_new), plan=plan, pos=pos, rows=tr)
        want, b = make()
        at = tr.long().expand(Bn, -1)
        # in the same layout: rows in another one take a kernel that may contract a fp32 sum differently
        pick = lambda x: _dev(_np(torch.stack([x[i][:, at[i]] for i in range(Bn)])), dtype, layout)  # noqa: E731
        ps = torch.stack([pos[0, i, at[i]] for i in range(Bn)])[None].contiguous() if rotated else None
        want.append(pick(kn), pick(vn), _i32(start), None if n_new is None else _i32(n_new), plan=plan, pos=ps)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    got, a = make()
    keep = [x.clone() for x in a]
    got.append(kn, vn, _i32([0, 0, 0]), plan=plan, pos=pos, rows=_i32([[30, -1], [2 ** 31 - 1, -2 ** 31], [99, 30]]))
    assert all(torch.equal(x, y) for x, y in zip(a, keep))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("kind", ["f32", "bf16", "8"])
@pytest.mark.parametrize("layout", ["bhnd", "odd"])
def test_read(lib, kind, d, layout):
    """Positions in order from plain and wrapped caches, 0 where the cache does not hold one, in
    both types."""
    torch = _gpu()
    rng = np.random.default_rng(d)
    Bn, Hkv, cap, sinks, N = 5, 3, 21, 4, 40
    if kind == "8":
        c8 = Cache8(rng, Bn, Hkv, cap, d, 15, sinks, layout)
        c, vals = c8.cache, c8.vals
    else:
        vals = [_draw(rng, (Bn, Hkv, cap, d), kind).astype(np.float64) for _ in range(2)]
        c = B.WinCache(*(_dev(x, kind, layout) for x in vals), 15, sinks)
    first, lens = [0, -3, 990, 5, 2 ** 31 - 20], [21, 9, 1000, 0, 2 ** 31 - 1]
    want = [np.zeros((Bn, Hkv, N, d)) for _ in range(2)]
    for b in range(Bn):
        for p, s in zip(*([x.tolist() for x in T.slots_held(lens[b], cap, sinks)] if lens[b] < 2000 else
                          (range(2 ** 31 - 1 - (cap - sinks), 2 ** 31 - 1),
                           [W.slot(p, cap, sinks) for p in range(2 ** 31 - 1 - (cap - sinks), 2 ** 31 - 1)]))):
            if first[b] <= p < first[b] + N:
                for w, x in zip(want, vals):
                    w[b, :, p - first[b]] = x[b, :, s]
    for dt in (torch.float32, torch.bfloat16):
        got = c.read(_i32(first), N, _i32(lens), dtype=dt)
        for g, w in zip(got, want):
            assert g.dtype == dt and g.shape == (Bn, Hkv, N, d)
            assert np.array_equal(_np(g), _np(torch.from_numpy(w).to(dt)))
    big = torch.full((2, Bn, N, Hkv, d + 1), 7.0, device="cuda")       # token-major rows of d + 1
    out = [x.transpose(1, 2)[..., :d] for x in big]
    got = c.read(_i32(first), N, _i32(lens), out_k=out[0], out_v=out[1])
    assert got[0] is out[0] and all(np.array_equal(_np(g), w) for g, w in zip(out, want)) and (big[..., d] == 7.0).all()


# ---------------------------------------------------------------- GPU: attention
DECODES = [
    # Bn, Hq, Hkv, cap, window, sinks, lens
    (1, 1, 1, 1, 1, 0, [1]), (3, 2, 2, 9, 7, 2, [0, 1, 5]), (2, 4, 1, 9, 7, 2, [9, 1000]), (2, 7, 1, 40, 33, 4, [37, 12345]),
    (1, 8, 1, 300, 290, 4, [2000000000]), (4, 16, 2, 140, 128, 0, [-3, 64, 128, 129]), (1, 2, 2, 700, 600, 64, [650]),
    (2, 32, 1, 1100, 1024, 4, [1028, 5000]), (16, 8, 8, 257, 200, 1, list(range(100, 260, 10))), (1, 65, 1, 130, 100, 2, [500]),
    (1, 4, 1, 40000, 33000, 4, [39000]),
]


def _visible_slots(L, cap, window, sinks):
    L = max(L, 0)
    return {W.slot(p, cap, sinks) for p in list(range(min(sinks, L))) + list(range(max(L - window, 0), L))}


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", DECODES, ids=lambda s: "-".join(str(x) for x in s[:6]))
def test_decode_8bit(lib, size, dtype, d):
    """Wrapped and unwrapped caches, empty sequences, NaN in every slot that is not visible."""
    torch = _gpu()
    Bn, Hq, Hkv, cap, window, sinks, lens = size
    rng = np.random.default_rng(cap + Hq)
    c = Cache8(rng, Bn, Hkv, cap, d, window, sinks)
    c.hide(lambda b: _visible_slots(lens[b], cap, window, sinks))
    q = _draw(rng, (Bn, Hq, d), dtype)
    tq = _dev(q[:, :, None], dtype, "bhnd")[:, :, 0]
    lse = torch.empty((Bn, Hq), device="cuda")
    o = c.cache.decode(tq, _i32(lens), 1 / math.sqrt(d), lse=lse)
    B.psa_attn_sync_status()
    if max(lens) > 1 << 20:                                   # the same slots at a smaller length
        lens = [x - (x - 4 * cap) // (cap - sinks) * (cap - sinks) for x in lens]
    ref = T.tree(q[:, :, None].astype(np.float64), *c.vals, None, None, lens, None, None, cap, window, sinks, 1 / math.sqrt(d),
                 W.U[dtype], c.scales[1])
    _close(o[:, :, None], ref[0], ref[2], "O")
    _close(lse[..., None], ref[1], ref[3], "LSE")
    assert torch.equal(o, c.cache.decode(tq, _i32(size[-1]), 1 / math.sqrt(d)))


def _tree_parents(rng, Bn, n, kind):
    if kind == "run":
        return None
    if kind == "chain":
        return np.tile(np.arange(-1, n - 1), (Bn, 1)).astype(np.int32)
    if kind == "star":                                        # every node a root
        return np.full((Bn, n), -1, dtype=np.int32)
    p = np.stack([[int(rng.integers(max(-1, t - 6), t)) for t in range(n)] for _ in range(Bn)]).astype(np.int32)
    if kind == "wild":                                        # values that name no earlier node
        p[:, ::3] = rng.choice([-2 ** 31, -7, n, 2 ** 31 - 1], size=p[:, ::3].shape)
        p[:, 1::5] = np.arange(n)[1::5]
    return p


TREES = [
    # Bn, Hq, Hkv, T, cap, window, sinks, lens, n_new, parents
    (1, 1, 1, 1, 1, 1, 0, [1], None, "run"),
    (3, 2, 2, 3, 9, 7, 2, [0, 1, 5], None, "tree"),
    (2, 4, 1, 5, 9, 7, 2, [9, 1000], [5, 2], "tree"),
    (2, 7, 1, 9, 40, 33, 4, [37, 12345], None, "wild"),
    (2, 4, 2, 16, 160, 150, 4, [70, 500], None, "star"),
    (2, 4, 2, 17, 50, 9, 3, [44, 1000], [17, 11], "chain"),           # paths longer than the window
    (1, 2, 1, 40, 12, 5, 6, [3], None, "run"),                        # sinks among the drafts
    (4, 16, 2, 8, 140, 128, 0, [-3, 64, 128, 129], [8, 0, 3, 99], "tree"),
    (1, 8, 4, 33, 700, 600, 64, [650], None, "tree"),
    (2, 32, 2, 26, 1100, 1024, 4, [1028, 5000], [26, 20], "tree"),
    (1, 2, 2, 256, 300, 290, 4, [1000], None, "tree"),
    (1, 8, 1, 200, 520, 500, 0, [511], [199], "run"),
    (1, 4, 1, 12, 9000, 8192, 17, [8999], None, "tree"),
    (2, 6, 3, 64, 290, 257, 2, [280, 5000], None, "tree"),
    (1, 24, 2, 11, 64, 50, 2, [33], None, "tree"),
    (2, 2, 1, 4, 70, 60, 2, [66, 900], [4, 3], "tree"),               # up to 8 rows
    (1, 8, 1, 1, 400, 380, 4, [1000], None, "run"),
    (1, 3, 3, 7, 12, 5, 2, [11], None, "chain"),
]
KINDS = [("f32", False), ("bf16", False), ("f32", True), ("bf16", True)]


class Tree:
    def __init__(self, dtype, is8, d, Bn, Hq, Hkv, n, cap, window, sinks, lens, n_new, parents, layout="bnhd", seed=0, std=1.0,
                 garbage=True):
        rng = np.random.default_rng(900 + seed + n)
        self.dtype, self.size, self.lens, self.n_new = dtype, (cap, window, sinks), lens, n_new
        self.scale = 1 / math.sqrt(d)
        if is8:
            c = Cache8(rng, Bn, Hkv, cap, d, window, sinks, "bhnd" if layout in ("bnhd", "bhnd") else "odd", std)
            self.vals, self.vs, self.cache = c.vals, c.scales[1], c.cache
            if garbage:
                c.hide(lambda b: self._seen(b))
        else:
            self.vals, self.vs = [_draw(rng, (Bn, Hkv, cap, d), dtype, std).astype(np.float64) for _ in range(2)], None
            dirty = [x.copy() for x in self.vals]
            if garbage:
                for b in range(Bn):
                    seen = self._seen(b)
                    hidden = [s for s in range(cap) if s not in seen]
                    dirty[0][b, :, hidden], dirty[1][b, :, hidden] = np.nan, np.inf
            self.cache = B.WinCache(*(_dev(x, dtype, "bhnd" if layout == "bnhd" else layout) for x in dirty), window, sinks)
        self.x = [_draw(rng, (Bn, h, n, d), dtype, std).astype(np.float64) for h in (Hq, Hkv, Hkv)]
        self.real = [n] * Bn if n_new is None else [min(max(x, 0), n) for x in n_new]
        if garbage:
            for b in range(Bn):
                for x in self.x:
                    x[b, :, self.real[b]:] = np.nan
        self.t = [_dev(x, dtype, layout) for x in self.x]
        self.parents = _tree_parents(rng, Bn, n, parents)

    def _seen(self, b):
        cap, window, sinks = self.size
        return _visible_slots(self.lens[b], cap, window, sinks)

    def args(self):
        return dict(parents=None if self.parents is None else _i32(self.parents.tolist()),
                    n_new=None if self.n_new is None else _i32(self.n_new))

    def run(self, algo=0, **kw):
        return self.cache.tree(*self.t, _i32(self.lens), self.scale, algo=algo, **self.args(), **kw)

    def check(self, algo=0):
        torch = _gpu()
        q, kn, vn = self.x
        lse = torch.empty(q.shape[:3], device="cuda")
        o = self.run(algo, lse=lse)
        B.psa_attn_sync_status()
        cap, window, sinks = self.size
        ref = T.tree(q, *self.vals, kn, vn, self.lens, self.real, self.parents, cap, window, sinks, self.scale, W.U[self.dtype],
                     self.vs)
        _close(o, ref[0], ref[2], "O")
        _close(lse, ref[1], ref[3], "LSE")
        assert torch.equal(o, self.run(algo))
        return o


ALGOS = [(k, a) for k in KINDS for a in ((B.PSA_ALGO_SIMT, B.PSA_ALGO_TC) if k[0] == "bf16" else (B.PSA_ALGO_AUTO,))]


def _name(x):
    kind, algo = x if isinstance(x[0], tuple) else (x, 0)
    return kind[0] + ("-8" if kind[1] else "") + ("-tc" if algo == B.PSA_ALGO_TC else "")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("kind", ALGOS, ids=_name)
@pytest.mark.parametrize("size", TREES, ids=lambda s: "-".join(str(x) for x in s[:7]))
def test_tree(lib, size, kind, d):
    """NaN in every slot that no node sees and in padding rows; rows beyond n_new come out as 0
    (LSE -inf)."""
    _gpu()
    c = Tree(*kind[0], d, *size, seed=d)
    o = c.check(kind[1])
    for b, n in enumerate(c.real):
        assert (o[b, :, n:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS, ids=_name)
@pytest.mark.parametrize("layout", ["bhnd", "chan", "odd"])
@pytest.mark.parametrize("n", [7, 60])
def test_tree_layouts(lib, kind, layout, n):
    torch = _gpu()
    if layout == "chan" and not kind[1]:
        pytest.skip("a cache's features are adjacent")
    c = Tree(*kind, 64, 2, 8, 2, n, 90, 70, 3, [55, 400], [n, n - 3], "tree", layout=layout)
    o = c.check()
    out = torch.full((2, n, 8, 72), 3.0, dtype=o.dtype, device="cuda")           # token-major, wider rows
    c.run(out=out.transpose(1, 2)[..., :64])
    assert torch.equal(out.transpose(1, 2)[..., :64], o) and (out[..., 64:] == 3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ALGOS, ids=_name)
def test_tree_large_scores(lib, kind):
    """Scores of several hundred; values whose rows differ by factors of up to e^4."""
    _gpu()
    Tree(*kind[0], 64, 2, 4, 2, 20, 300, 280, 4, [290, 1000], None, "tree", std=8.0).check(kind[1])


MORE_TREES = [
    # many sequences, some without tokens or without a cache, so that a block has several items and an
    # item several blocks; a run's end and start inside a tile; two row tiles and more
    (70, 2, 1, 70, 300, 260, 3, [0, 1, 2, 130, 259, 262, 263, 1000, 299, 5000] * 7, [70, 0, 1, 64, 65, 33, 70, 70, 2, 69] * 7, "tree"),
    (1, 2, 2, 64, 20000, 19000, 4, [19990], None, "tree"),
    (3, 4, 1, 130, 700, 650, 5, [690, 20, 100000], [130, 129, 7], "chain"),
    (2, 9, 1, 100, 520, 512, 8, [1000, 513], [100, 90], "wild"),
    (1, 128, 1, 5, 200, 150, 2, [170], None, "tree"),
    (400, 1, 1, 2, 40, 30, 1, [x % 90 for x in range(400)], [x % 3 for x in range(400)], "tree"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [a for a in ALGOS if a[0][0] == "bf16"], ids=_name)
@pytest.mark.parametrize("size", MORE_TREES, ids=lambda s: "-".join(str(x) for x in s[:7]))
def test_tree_work_shared_by_blocks(lib, size, kind):
    _gpu()
    Tree(*kind[0], 64, *size, seed=3).check(kind[1])


@pytest.mark.gpu
def test_tree_tc_refuses(lib):
    """Layouts and types that the tensor-core kernel does not take."""
    torch = _gpu()
    for kind, layout in ((("bf16", False), "odd"), (("f32", False), "bnhd"), (("bf16", True), "chan")):
        c = Tree(*kind, 64, 2, 8, 2, 9, 90, 70, 3, [55, 400], None, "tree", layout=layout, garbage=False)
        with pytest.raises(B.PsaError) as e:
            c.run(B.PSA_ALGO_TC)
        assert e.value.code == B.PSA_ERR_UNSUPPORTED
        c.run()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_8bit_values_of_very_different_sizes(lib, dtype):
    """Rows of 2^-60 next to rows of 2^60: the output is as near as the bounds say to the weighted
    sum, also where the heavy keys have the small values."""
    torch = _gpu()
    rng = np.random.default_rng(77)
    c = Cache8(rng, 1, 1, 200, 64, 190, 4)
    up = 2.0 ** rng.choice([-60.0, 0.0, 60.0], size=200)
    up[:64] = 2.0 ** -60
    c.vals[1] *= up[None, None, :, None]
    c.scales[1] *= up[None, None]
    c.vs.copy_(torch.from_numpy(c.scales[1]).float())
    q = _draw(rng, (1, 4, 64), dtype)
    q[0, 0] = 30 * c.vals[0][0, 0, 5] / np.abs(c.vals[0][0, 0, 5]).max()          # one heavy key with small values
    q = round_storage(q, dtype)
    for L in (64, 150):
        o = c.cache.decode(_dev(q[:, :, None], dtype)[:, :, 0], _i32([L]), 0.125)
        ref = T.tree(q[:, :, None].astype(np.float64), *c.vals, None, None, [L], None, None, 200, 190, 4, 0.125, W.U[dtype],
                     c.scales[1])
        _close(o[:, :, None], ref[0], ref[2], f"L={L}")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [a for a in ALGOS if a[0][1]], ids=_name)
@pytest.mark.parametrize("size", [(3, 4, 2, 7, 300, 260, 3, [290, 100, 1000], [7, 5, 7], "tree"), (2, 32, 1, 9, 400, 390, 2, [390, 777], None, "chain")],
                         ids=["small", "rows"])
def test_8bit_scales_that_no_write_makes(lib, kind, size):
    """Scales 3 or 5 times a power of two (times a code of 4 bits they still fit bf16, so that the
    bounds hold as they are), and zero: for single rows, and for all values of a sequence."""
    torch = _gpu()
    c = Tree(*kind[0], 64, *size, seed=11, garbage=False)
    rng = np.random.default_rng(12)
    for i, to in enumerate((c.cache.k_scale, c.cache.v_scale)):
        s = to.double().cpu().numpy()
        by = rng.choice([3.0, 5.0, 1.0, 0.0], size=s.shape)
        if i:
            by[1] = 0.0
        c.vals[i] *= by[..., None]
        to.copy_(torch.from_numpy(s * by).float())
        if i:
            c.vs = s * by
    c.check(kind[1])
    lens = _i32(c.lens)
    q = c.t[0][:, :, 0].contiguous()
    o = c.cache.decode(q, lens, c.scale)
    ref = T.tree(c.x[0][:, :, :1], *c.vals, None, None, c.lens, None, None, *c.size, c.scale, W.U[c.dtype], c.vs)
    _close(o[:, :, None], ref[0], ref[2], "decode")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ALGOS, ids=_name)
def test_tree_key_of_nan_stays_with_its_rows(lib, kind):
    """A key that is NaN reaches the nodes that see it and no other: the oldest cached key of a
    root's window, and a draft's key, which its descendants see."""
    torch = _gpu()
    L, window, n = 100, 40, 9
    c = Tree(*kind[0], 64, 1, 4, 2, n, 128, window, 0, [L], None, "tree", seed=5, garbage=False)
    want = c.run(kind[1])
    c.parents = np.array([[-1, 0, 1, -1, 3, 3, 5, 2, 4]])
    want = c.run(kind[1])
    line = T.ancestors(c.parents[0], n)
    at = W.slot(L - window + 1, 128, 0)
    if kind[0][1]:
        c.cache.k_scale[0, :, at] = float("nan")
    else:
        c.cache.k[0, :, at] = float("nan")
    c.t[1][:, :, 5] = float("nan")
    got = c.run(kind[1])
    B.psa_attn_sync_status()
    hit = (line.sum(-1) == 1) | line[:, 5]
    assert torch.isnan(got[0, :, hit]).all() and torch.equal(got[0, :, ~hit], want[0, :, ~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS, ids=_name)
def test_tree_in_graphs_and_on_two_streams(lib, kind):
    """Captured and replayed on new lengths and trees; two caches at once on two streams."""
    torch = _gpu()
    cases = [Tree(*kind, 128, 2, 8, 2, 40, 2100, 2048, 4, [2000, 5000], None, "tree", seed=s, garbage=False) for s in (1, 2)]
    args = [(c.t, _i32(c.lens), _i32(c.parents.tolist()), _i32([40, 33])) for c in cases]
    run = lambda c, a: c.cache.tree(*a[0], a[1], c.scale, parents=a[2], n_new=a[3])  # noqa: E731
    want = [run(c, a) for c, a in zip(cases, args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(12):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(cases[i], args[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(w, x) for w, g in zip(want, got) for x in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = run(cases[0], args[0])
    args[0][1].copy_(_i32([7, 900]))
    args[0][2].copy_(torch.roll(args[0][2], 1, 0))
    args[0][3].copy_(_i32([1, 40]))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, run(cases[0], args[0]))


@pytest.mark.gpu
@pytest.mark.parametrize("is8", [False, True])
def test_tree_and_store_past_32_bit_offsets(lib, is8):
    """A cache of 2^32 elements: slots whose element offsets pass 32 bits."""
    torch = _gpu()
    cap, d, n = 1 << 25, 128, 210
    g = torch.Generator(device="cuda").manual_seed(1)

    def make(cap):
        if not is8:
            return B.WinCache(*(torch.empty((1, 1, cap, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)), 200, 4)
        t = [torch.empty((1, 1, cap, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
        return B.WinCache(*t, 200, 4, *(torch.empty((1, 1, cap), device="cuda") for _ in range(2)))

    new = [torch.randn((1, 1, n, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    q, kn, vn = (torch.randn((1, h, 9, d), generator=g, device="cuda").to(torch.bfloat16) for h in (8, 1, 1))
    rows = torch.arange(n, dtype=torch.int32, device="cuda")
    out = []
    for c, start in ((make(cap), cap - n - 1), (make(400), 4 + 396 * 1000)):      # the same ring order of the rows
        c.append(new[0][:, :, :4], new[1][:, :, :4], _i32([0]))
        c.append(*new, _i32([start]), rows=rows)
        got = c.read(_i32([start]), n, _i32([start + n]))
        out.append((c.tree(q, kn, vn, _i32([start + n]), 0.1), c.decode(q[:, :, 0], _i32([start + n]), 0.1), *got))
        if not is8:
            assert torch.equal(got[0], new[0]) and torch.equal(got[1], new[1])
    for a, b in zip(*out):
        torch.testing.assert_close(a, b, rtol=2.0 ** -6, atol=2.0 ** -9)


# ---------------------------------------------------------------- together
@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS, ids=_name)
@pytest.mark.parametrize("capacity", [68, 400])
def test_speculative_serving(lib, kind, capacity):
    """Prompt, then trees of drafts whose accepted paths are appended, then single tokens: every
    accepted node's row is what the oracle says of the sequence that results.  Over 8-bit caches
    the oracle reads what read() gives of them."""
    torch = _gpu()
    dtype, is8 = kind
    rng = np.random.default_rng(51)
    Bn, Hq, Hkv, d, window, sinks, prompt, n = 2, 4, 2, 64, 60, 4, 90, 12
    scale, plan, u = 0.125, _plan(head_dim=d, sections=(32,)), W.U[dtype]
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    shape = (Bn, Hkv, capacity, d)
    if is8:
        cache = B.WinCache(*(torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in "kv"),
                           window, sinks, *(torch.full(shape[:3], float("nan"), device="cuda") for _ in "kv"))
    else:
        cache = B.WinCache(*(torch.full(shape, float("nan"), dtype=dt, device="cuda") for _ in "kv"), window, sinks)
    x = [_dev(_draw(rng, (Bn, Hkv, prompt, d), dtype), dtype) for _ in range(2)]
    pos = torch.arange(prompt, dtype=torch.int32, device="cuda")[None]
    cache.append(*x, _i32([0, 0]), n_new=_i32([prompt, prompt - 20]), plan=plan, pos=pos)
    lens = np.array([prompt, prompt - 20])

    def known(upto):
        """The cache's positions in order (zeros where it does not hold one)."""
        return [_np(t) for t in cache.read(_i32([0, 0]), int(max(upto)), _i32(upto.tolist()), dtype=torch.float32)]

    for step in range(4):
        parents = _tree_parents(rng, Bn, n, "tree")
        line = [T.ancestors(p, n) for p in parents]
        depth = np.stack([a.sum(-1) - 1 for a in line])
        q, kn, vn = (_dev(_draw(rng, (Bn, h, n, d), dtype), dtype) for h in (Hq, Hkv, Hkv))
        p = _i32((lens[:, None] + depth)[None].tolist())
        q, kn = B.rope(plan, q, p, k=kn)
        o = cache.tree(q, kn, vn, _i32(lens.tolist()), scale, parents=_i32(parents.tolist()))
        k, v = known(lens)
        big = int(max(lens)) + 1                              # an oracle cache that slots positions in order
        pad = lambda t: np.pad(t, ((0, 0), (0, 0), (0, big - t.shape[2]), (0, 0)))  # noqa: E731
        ref = T.tree(_np(q), pad(k), pad(v), _np(kn), _np(vn), lens.tolist(), [n, n], parents, big, window, sinks, scale, u,
                     np.full((Bn, Hkv, big), np.abs(v).max() / 224) if is8 else None)
        _close(o, ref[0], ref[2], f"step {step}")
        leaf = [int(np.argmax(x)) for x in depth]
        path = [np.nonzero(a[t])[0].tolist() for a, t in zip(line, leaf)]
        m = max(len(x) for x in path)
        cache.append(kn, vn, _i32(lens.tolist()), n_new=_i32([len(x) for x in path]),
                     rows=_i32([x + [-1] * (m - len(x)) for x in path]))
        lens = lens + [len(x) for x in path]
        # the newest token alone gives the leaf's row, up to its key and value in 8 bits
        last = torch.stack([q[b, :, t] for b, t in enumerate(leaf)])
        got = cache.decode(last, _i32(lens.tolist()), scale)
        k, v = known(lens)
        r = [[W.attention(_np(last)[b, h][None], k[b, h // 2, :lens[b]], v[b, h // 2, :lens[b]], scale, window, sinks, u)
              for h in range(Hq)] for b in range(Bn)]
        want, bound = (np.array([[x[i][0] for x in heads] for heads in r]) for i in (0, 2))
        # what fp16's small numbers lose over an 8-bit cache: see tree_oracle
        extra = 2.0 ** -25 * 448 * max(lens) * np.abs(v).max() / 224 if is8 and dtype == "bf16" else 0.0
        _close(got, want, bound + extra, f"token after step {step}")
