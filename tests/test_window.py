"""Sliding-window attention with sinks (forward, backward), rotary positions with
several axes, the rolling cache and its single-token attention: refusals and the
oracle's own checks on the CPU; on the GPU, every operator against the oracle
within the bounds that it derives, and runs of them together."""
import ctypes
import math

import numpy as np
import pytest

import window_oracle as W
from self_attention_backward_gb300 import binding as B
from self_attention_backward_gb300.inputs import round_storage

FAKE = 0x10000
INF = float("inf")


@pytest.fixture(scope="module")
def lib():
    from self_attention_backward_gb300.build import build
    build()
    return B.lib()


# ---------------------------------------------------------------- the oracle itself
def test_oracle_gradient_matches_differences():
    rng = np.random.default_rng(5)
    q, k, v, do = rng.normal(size=(6, 4)), rng.normal(size=(9, 4)), rng.normal(size=(9, 4)), rng.normal(size=(6, 4))
    args = (0.7, 3, 2)
    o, lse, _, _ = W.attention(q, k, v, *args)
    got = W.gradient(q, k, v, o, lse, do, *args)[:3]
    loss = lambda: (W.attention(q, k, v, *args)[0] * do).sum()  # noqa: E731
    for x, g in zip((q, k, v), got):
        for at in np.ndindex(x.shape):
            keep, h = x[at], 1e-6
            x[at] = keep + h
            up = loss()
            x[at] = keep - h
            down = loss()
            x[at] = keep
            assert abs((up - down) / (2 * h) - g[at]) < 1e-7


def test_oracle_mask():
    see = W.visible(3, 8, window=2, sinks=1)
    assert see.astype(int).tolist() == [[1, 0, 0, 0, 1, 1, 0, 0], [1, 0, 0, 0, 0, 1, 1, 0], [1, 0, 0, 0, 0, 0, 1, 1]]
    assert not W.visible(5, 2, 4, 1)[:3].any()          # more rows than keys: the first see nothing
    assert W.visible(4, 4, 100, 0).sum() == 10


def test_oracle_slots():
    assert [W.slot(p, 5, 2) for p in range(9)] == [0, 1, 2, 3, 4, 2, 3, 4, 2]


# ---------------------------------------------------------------- refusals (nothing is launched)
def _shape(**kw):
    a = dict(B=1, q_heads=4, kv_heads=2, Nq=8, Nk=8, head_dim=32, window=4, sinks=1, scale=0.5, dtype=B.PSA_BF16)
    a.update(kw)
    return B.psa_win_shape(*a.values())


def _view(base=FAKE, sb=4 * 8 * 32, sh=8 * 32, sn=32, sj=1):
    return B.psa_attn_view(base, sb, sh, sn, sj)


def _fwd(lib, shape=None, lse=FAKE, q_lens=None, algo=0, **views):
    v = dict(q=_view(), k=_view(), v=_view(), o=_view())
    v.update(views)
    return lib.psa_win_attn_fwd(_shape() if shape is None else shape, v["q"], v["k"], v["v"], v["o"], lse, q_lens, None,
                                algo, None)


BAD_SHAPES = [
    (dict(head_dim=48), B.PSA_ERR_UNSUPPORTED), (dict(head_dim=256), B.PSA_ERR_UNSUPPORTED),
    (dict(window=0), B.PSA_ERR_ARG), (dict(window=-3), B.PSA_ERR_ARG), (dict(sinks=-1), B.PSA_ERR_ARG),
    (dict(q_heads=3), B.PSA_ERR_ARG), (dict(kv_heads=0), B.PSA_ERR_ARG), (dict(Nq=-1), B.PSA_ERR_ARG),
    (dict(B=-1), B.PSA_ERR_ARG), (dict(dtype=5), B.PSA_ERR_ARG), (dict(scale=float("nan")), B.PSA_ERR_ARG),
    (dict(scale=INF), B.PSA_ERR_ARG), (dict(B=1 << 20, Nk=1 << 20, q_heads=64, kv_heads=64), B.PSA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_SHAPES)
def test_attention_refuses_shapes(lib, kw, code):
    assert _fwd(lib, _shape(**kw)) == code
    assert B.psa_attn_last_error()
    assert lib.psa_win_attn_bwd_workspace_bytes(_shape(**kw)) == 0
    v = _view()
    assert lib.psa_win_attn_bwd(_shape(**kw), v, v, v, v, FAKE, v, v, v, v, None, None, FAKE, 1 << 40, 0, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), B.PSA_ERR_ARG), (dict(k=_view(0)), B.PSA_ERR_ARG), (dict(o=_view(FAKE + 8)), B.PSA_ERR_ALIGN),
    (dict(v=_view(sn=-32)), B.PSA_ERR_ARG), (dict(o=_view(sn=0)), B.PSA_ERR_ARG), (dict(lse=None), B.PSA_ERR_ARG),
    (dict(lse=FAKE + 4), B.PSA_ERR_ALIGN), (dict(q_lens=FAKE + 2), B.PSA_ERR_ALIGN), (dict(algo=3), B.PSA_ERR_ARG),
    (dict(k=_view(sh=1 << 41)), B.PSA_ERR_UNSUPPORTED), (dict(shape=_shape(dtype=B.PSA_F32), algo=B.PSA_ALGO_TC),
                                                         B.PSA_ERR_UNSUPPORTED),
    (dict(q=_view(sj=2, sn=64), algo=B.PSA_ALGO_TC), B.PSA_ERR_UNSUPPORTED),
    (dict(k=_view(sn=36), algo=B.PSA_ALGO_TC), B.PSA_ERR_UNSUPPORTED),
    (dict(v=_view(sh=0), algo=B.PSA_ALGO_TC), B.PSA_ERR_UNSUPPORTED),
])
def test_attention_refuses_tensors(lib, kw, code):
    assert _fwd(lib, **kw) == code


def test_attention_empty_calls(lib):
    for kw in (dict(B=0), dict(q_heads=0, kv_heads=0), dict(Nq=0)):
        assert lib.psa_win_attn_fwd(_shape(**kw), None, None, None, None, None, None, None, 0, None) == B.PSA_OK
    v = [None] * 4
    for kw in (dict(B=0), dict(Nq=0, Nk=0)):
        assert lib.psa_win_attn_bwd(_shape(**kw), *v, None, *v, None, None, None, 0, 0, None) == B.PSA_OK
        assert lib.psa_win_attn_bwd_workspace_bytes(_shape(**kw)) == 0


def test_backward_refuses(lib):
    v = _view()
    need = lib.psa_win_attn_bwd_workspace_bytes(_shape())
    assert need >= 4 * 8 * 4
    call = lambda dk=v, ws=FAKE, n=need, d_o=v: lib.psa_win_attn_bwd(  # noqa: E731
        _shape(), v, v, v, v, FAKE, d_o, v, dk, v, None, None, ws, n, 0, None)
    assert call(n=need - 1) == B.PSA_ERR_WORKSPACE
    assert call(ws=None) == B.PSA_ERR_WORKSPACE
    assert call(ws=FAKE + 4) == B.PSA_ERR_ALIGN
    assert call(dk=_view(sb=0, sh=0)) == B.PSA_ERR_ARG
    assert call(d_o=None) == B.PSA_ERR_ARG


def test_workspace_covers_the_sink_sums(lib):
    """24 bytes of row statistics, for whole 128-row tiles, for short sequences; with sinks and a long
    sequence the partial sums too, and no more of them than 64 chunks."""
    d_only = lambda s: 24 * s.B * s.q_heads * ((s.Nq + 127) // 128 * 128)  # noqa: E731
    for kw in (dict(), dict(Nq=900, Nk=900), dict(Nq=5000, Nk=5000, sinks=0), dict(Nq=5000, Nk=5000, window=4900)):
        s = _shape(**kw)
        assert lib.psa_win_attn_bwd_workspace_bytes(s) == d_only(s)
    for n in (5000, 1 << 20):
        s = _shape(Nq=n, Nk=n, sinks=3)
        parts = lib.psa_win_attn_bwd_workspace_bytes(s) - d_only(s)
        per = 2 * 2 * 3 * 32 * 4
        assert parts % per == 0 and 2 < parts // per <= 65


def _plan(**kw):
    a = dict(head_dim=32, sections=(16,), theta=10000.0, rot_dim=None, ladder=0, interleaved=False)
    a.update(kw)
    return B.RopePlan(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=48), B.PSA_ERR_UNSUPPORTED), (dict(rot_dim=33), B.PSA_ERR_ARG), (dict(rot_dim=34), B.PSA_ERR_ARG),
    (dict(rot_dim=0), B.PSA_ERR_ARG), (dict(sections=(8,)), B.PSA_ERR_ARG), (dict(sections=(17, -1)), B.PSA_ERR_ARG),
    (dict(sections=()), B.PSA_ERR_ARG), (dict(sections=(4, 4, 4, 4)), B.PSA_ERR_ARG), (dict(theta=1.0), B.PSA_ERR_ARG),
    (dict(theta=float("nan")), B.PSA_ERR_ARG), (dict(ladder=2), B.PSA_ERR_ARG),
])
def test_plan_refuses(lib, kw, code):
    with pytest.raises(B.PsaError) as e:
        _plan(**kw)
    assert e.value.code == code


def test_plan_frequencies(lib):
    """The turn fractions are the frequencies / 2 pi to double precision, section by section."""
    p = _plan(sections=(4, 6, 6), theta=500.0).c
    want = 500.0 ** -(np.arange(16) / 16) / (2 * math.pi)
    np.testing.assert_allclose(np.array(p.turn[:16], dtype=np.float64) / 2.0 ** 64, want, rtol=1e-14)
    assert list(p.axis[:16]) == [0] * 4 + [1] * 6 + [2] * 6
    p = _plan(sections=(10, 6), ladder=B.PSA_ROPE_PER_AXIS).c
    want = np.concatenate([10000.0 ** -(np.arange(s) / s) for s in (10, 6)]) / (2 * math.pi)
    np.testing.assert_allclose(np.array(p.turn[:16], dtype=np.float64) / 2.0 ** 64, want, rtol=1e-14)


def test_rope_refuses(lib):
    p, v = _plan().c, _view()
    call = lambda plan=p, x=v, y=v, x2=None, y2=None, heads=4, pos=FAKE, pa=0, pb=0, n=8, dt=B.PSA_F32: lib.psa_rope(  # noqa: E731
        plan, x, y, heads, x2, y2, 2, 1, n, pos, pa, pb, 0, dt, None)
    assert call(plan=None) == B.PSA_ERR_ARG
    assert call(plan=B.psa_rope_plan()) == B.PSA_ERR_ARG
    assert call(x=None) == B.PSA_ERR_ARG
    assert call(x2=v) == B.PSA_ERR_ARG
    assert call(pos=None) == B.PSA_ERR_ARG
    assert call(pos=FAKE + 1) == B.PSA_ERR_ALIGN
    assert call(pb=-1) == B.PSA_ERR_ARG
    assert call(heads=-1) == B.PSA_ERR_ARG
    assert call(dt=9) == B.PSA_ERR_ARG
    assert call(y=_view(FAKE + 4)) == B.PSA_ERR_ALIGN
    assert call(y=_view(sh=0)) == B.PSA_ERR_ARG
    assert call(n=0, x=None, pos=None) == B.PSA_OK


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE * 16, B=1, kv_heads=2, capacity=8, head_dim=32, window=4, sinks=1, dtype=B.PSA_BF16,
             batch_stride=2 * 8 * 32, head_stride=8 * 32, slot_stride=32)
    a.update(kw)
    return B.psa_win_cache(*a.values())


BAD_CACHES = [
    (dict(capacity=4), B.PSA_ERR_ARG), (dict(window=0, capacity=1), B.PSA_ERR_ARG), (dict(sinks=-1), B.PSA_ERR_ARG),
    (dict(window=0x7fffffff, sinks=0x7fffffff), B.PSA_ERR_ARG), (dict(head_dim=8), B.PSA_ERR_UNSUPPORTED),
    (dict(dtype=3), B.PSA_ERR_ARG), (dict(k=None), B.PSA_ERR_ARG), (dict(v=FAKE + 8), B.PSA_ERR_ALIGN),
    (dict(v=FAKE), B.PSA_ERR_ARG), (dict(slot_stride=0), B.PSA_ERR_ARG), (dict(kv_heads=-1), B.PSA_ERR_ARG),
    (dict(head_stride=-8), B.PSA_ERR_ARG),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_cache_refuses(lib, kw, code):
    v = _view()
    assert lib.psa_win_cache_append(_cache(**kw), v, v, 8, FAKE, None, None, None, 0, 0, None) == code
    assert lib.psa_win_decode(_cache(**kw), v, v, None, 4, FAKE, 0.5, FAKE, 1 << 40, None) == code
    assert lib.psa_win_decode_workspace_bytes(_cache(**kw), 4) == 0


def test_append_and_decode_refuse(lib):
    v, c, p = _view(), _cache(), _plan().c
    app = lambda k=v, T=8, start=FAKE, n=None, plan=None, pos=None: lib.psa_win_cache_append(  # noqa: E731
        c, k, v, T, start, n, plan, pos, 0, 0, None)
    assert app(k=None) == B.PSA_ERR_ARG
    assert app(T=-1) == B.PSA_ERR_ARG
    assert app(start=None) == B.PSA_ERR_ARG
    assert app(n=FAKE + 2) == B.PSA_ERR_ALIGN
    assert app(plan=p) == B.PSA_ERR_ARG                      # a rotation without positions
    assert app(plan=_plan(head_dim=64, sections=(32,)).c, pos=FAKE) == B.PSA_ERR_ARG
    assert app(T=0, k=None, start=None) == B.PSA_OK
    dec = lambda q=v, o=v, heads=4, lens=FAKE, scale=0.5, lse=None: lib.psa_win_decode(  # noqa: E731
        c, q, o, lse, heads, lens, scale, FAKE, 1 << 40, None)
    assert dec(heads=3) == B.PSA_ERR_ARG
    assert dec(heads=0) == B.PSA_ERR_ARG
    assert dec(lens=None) == B.PSA_ERR_ARG
    assert dec(scale=INF) == B.PSA_ERR_ARG
    assert dec(q=None) == B.PSA_ERR_ARG
    assert dec(o=_view(sh=0)) == B.PSA_ERR_ARG
    assert dec(lse=FAKE + 2) == B.PSA_ERR_ALIGN
    need = lib.psa_win_decode_workspace_bytes(_cache(B=1, capacity=1 << 20, window=1 << 19, batch_stride=1 << 26,
                                                     head_stride=1 << 25), 4)
    if need:
        big = _cache(capacity=1 << 20, window=1 << 19, batch_stride=1 << 26, head_stride=1 << 25)
        assert lib.psa_win_decode(big, v, v, None, 4, FAKE, 0.5, FAKE, need - 1, None) == B.PSA_ERR_WORKSPACE
        assert lib.psa_win_decode(big, v, v, None, 4, FAKE, 0.5, None, need, None) == B.PSA_ERR_WORKSPACE


def test_binding_refuses_mismatched_tensors(lib):
    torch = pytest.importorskip("torch")
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    q, k = z(1, 4, 8, 32), z(1, 2, 8, 32)
    bad = [
        lambda: B.win_attn_fwd(q[0], k, k, 1.0, 4, 0),
        lambda: B.win_attn_fwd(q, k, z(1, 2, 9, 32), 1.0, 4, 0),
        lambda: B.win_attn_fwd(q, k, k.float(), 1.0, 4, 0),
        lambda: B.win_attn_fwd(q, k, k, 1.0, 4, 0, kv_lens=z(1, t=torch.int64)),
        lambda: B.win_attn_fwd(q, k, k, 1.0, 4, 0, kv_lens=z(2, t=torch.int32)),
        lambda: B.win_attn_fwd(q, k, k, 1.0, 4, 0),                            # not on a GPU
        lambda: B.win_attn_bwd(q, k, k, q, z(1, 4, 8), q, 1.0, 4, 0),          # lse in bf16
        lambda: B.rope(_plan(), q, z(2, 1, 8, t=torch.int32)),
        lambda: B.rope(_plan(), z(1, 4, 8, 64), z(1, 1, 8, t=torch.int32)),
        lambda: B.WinCache(k, k[..., :16], 4, 1),
        lambda: B.WinCache(k.transpose(2, 3), k.transpose(2, 3), 4, 1),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- GPU
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


def _draw(rng, shape, dtype, std=1.0):
    return round_storage(rng.normal(0.0, std, size=shape), dtype)


def _dev(x, dtype, layout="bnhd"):
    """x [B, H, N, d] on the GPU: token-major memory, head-major, or with odd strides."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda().to({"bf16": torch.bfloat16, "f32": torch.float32}[dtype])
    if layout == "bnhd":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "bhnd":
        return t.contiguous()
    if layout == "chan":                                    # channel-major: [B, H, d, N]
        return t.transpose(2, 3).contiguous().transpose(2, 3)
    Bn, H, N, d = t.shape                                   # rows of d + 3 elements
    big = torch.full((Bn, H, N, d + 3), float("nan"), dtype=t.dtype, device="cuda")
    big[..., :d] = t
    return big[..., :d]


def _np(t):
    return t.double().cpu().numpy()


def _close(got, ref, bound, what):
    """Within the derived bound, infinities in the same places."""
    got = _np(got) if not isinstance(got, np.ndarray) else got
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin]), what
    err = np.abs(got - ref)[fin]
    over = err > bound[fin] + 1e-30
    assert not over.any(), (what, float((err[over] / (bound[fin][over] + 1e-30)).max()), int(over.sum()))


class Case:
    def __init__(self, dtype, d, Bn, Hq, Hkv, Nq, Nk, window, sinks, q_lens=None, kv_lens=None, layout="bnhd", seed=0, std=1.0,
                 garbage=False):
        rng = np.random.default_rng(7000 + seed)
        self.dtype, self.window, self.sinks, self.scale = dtype, window, sinks, 1 / math.sqrt(d)
        self.q, self.do = (_draw(rng, (Bn, Hq, Nq, d), dtype, std) for _ in range(2))
        self.k, self.v = (_draw(rng, (Bn, Hkv, Nk, d), dtype, std) for _ in range(2))
        self.ql, self.kl = q_lens, kv_lens
        clamp = lambda l, n: [n] * Bn if l is None else [min(max(x, 0), n) for x in l]  # noqa: E731
        self.qn, self.kn = clamp(q_lens, Nq), clamp(kv_lens, Nk)
        if garbage:                                          # padding holds anything
            for b in range(Bn):
                self.q[b, :, self.qn[b]:] = np.nan
                self.do[b, :, self.qn[b]:] = np.inf
                self.k[b, :, self.kn[b]:] = np.nan
                self.v[b, :, self.kn[b]:] = -np.inf
        self.t = [_dev(x, dtype, layout) for x in (self.q, self.k, self.v, self.do)]

    def lens(self):
        import torch
        f = lambda l: None if l is None else torch.tensor(l, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(q_lens=f(self.ql), kv_lens=f(self.kl))

    def forward(self, algo=0):
        q, k, v, _ = self.t
        return B.win_attn_fwd(q, k, v, self.scale, self.window, self.sinks, algo=algo, **self.lens())

    def backward(self, o, lse, algo=0):
        q, k, v, do = self.t
        return B.win_attn_bwd(q, k, v, o, lse, do, self.scale, self.window, self.sinks, algo=algo, **self.lens())

    def check(self, algo=0):
        o, lse = self.forward(algo)
        B.psa_attn_sync_status()
        u = W.U[self.dtype]
        with np.errstate(invalid="ignore"):
            ref = W.batch_forward(*(x.astype(np.float64) for x in (self.q, self.k, self.v)), self.scale, self.window,
                                  self.sinks, self.qn, self.kn, u)
        _close(o, ref[0], ref[2], "O")
        _close(lse, ref[1], ref[3], "LSE")
        got = self.backward(o, lse, algo)
        B.psa_attn_sync_status()
        ref = W.batch_gradient(*(x.astype(np.float64) for x in (self.q, self.k, self.v)), _np(o), _np(lse),
                               self.do.astype(np.float64), self.scale, self.window, self.sinks, self.qn, self.kn, u)
        for name, g, r, bound in zip(("dQ", "dK", "dV"), got, ref[:3], ref[3:]):
            _close(g, r, bound, name)
        return o, lse, got


ALGOS = [("f32", B.PSA_ALGO_SIMT), ("bf16", B.PSA_ALGO_SIMT), ("bf16", B.PSA_ALGO_AUTO)]
SIZES = [
    # Bn, Hq, Hkv, Nq, Nk, window, sinks, q_lens, kv_lens
    (1, 1, 1, 1, 1, 1, 0, None, None),
    (2, 2, 1, 2, 2, 2, 0, None, None),
    (1, 2, 2, 63, 63, 7, 0, None, None),
    (1, 2, 1, 64, 64, 64, 4, None, None),
    (1, 1, 1, 65, 65, 1, 1, None, None),
    (2, 4, 2, 129, 129, 40, 3, None, None),
    (1, 3, 1, 200, 200, 500, 2, None, None),                 # the window covers everything
    (1, 2, 1, 257, 257, 33, 130, None, None),                # more than one tile of sinks
    (1, 2, 1, 300, 300, 10, 400, None, None),                # all keys are sinks
    (1, 2, 1, 5, 301, 64, 4, None, None),                    # the last rows of a long context
    (1, 2, 1, 130, 70, 20, 1, None, None),                   # more rows than keys
    (3, 2, 1, 150, 150, 50, 5, [150, 1, 64], [150, 1, 64]),  # a padded batch
    (4, 2, 2, 70, 140, 30, 2, [70, 0, 33, 9], [140, 50, 0, 5]),
    (1, 4, 1, 1500, 1500, 60, 4, None, None),                # far chunks of the sink rows
    (2, 2, 1, 1700, 1700, 100, 70, [1700, 900], [1700, 1300]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype,algo", ALGOS)
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "-".join(str(x) for x in s[:7]))
def test_attention(lib, size, dtype, algo, d):
    _gpu()
    if size[3] >= 1000 and d not in (64, 128):
        pytest.skip("long sequences at two head sizes")
    Case(dtype, d, *size, seed=d + size[3]).check(algo)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["bhnd", "chan", "odd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_layouts(lib, dtype, layout):
    """Head-major, channel-major and odd row strides; the outputs take the inputs' layout."""
    torch = _gpu()
    c = Case(dtype, 32, 2, 4, 2, 100, 100, 30, 2, layout=layout, seed=3)
    c.check()
    if layout == "odd":                                      # nothing outside the view is written
        q, k, v, do = c.t
        big = torch.full((2, 4, 100, 35), 7.0, dtype=q.dtype, device="cuda")
        o, _ = B.win_attn_fwd(q, k, v, c.scale, 30, 2, out=big[..., :32])
        assert (big[..., 32:] == 7.0).all() and torch.equal(o, c.forward()[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,algo", ALGOS)
@pytest.mark.parametrize("d", [64, 128])
def test_attention_padding_is_never_read(lib, dtype, algo, d):
    """NaN and infinities behind the sequences' ends reach nothing; padding rows come out as
    0 (LSE -inf), lengths outside their range are clamped."""
    torch = _gpu()
    c = Case(dtype, d, 4, 2, 1, 140, 200, 50, 3, q_lens=[140, 77, 0, 999], kv_lens=[130, 77, 200, -5], seed=11, garbage=True)
    o, lse, (dq, dk, dv) = c.check(algo)
    assert (o[1, :, 77:] == 0).all() and (lse[1, :, 77:] == -INF).all() and (dq[1, :, 77:] == 0).all()
    assert (dk[0, :, 130:] == 0).all() and (dv[3] == 0).all() and torch.isfinite(dk).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,algo", ALGOS)
def test_attention_large_scores(lib, dtype, algo):
    """Peaked softmax: scores of several hundred, where a plain exponential would overflow."""
    _gpu()
    Case(dtype, 64, 1, 2, 1, 200, 200, 90, 2, seed=5, std=8.0).check(algo)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-3])
@pytest.mark.parametrize("dtype,algo", ALGOS)
def test_attention_scales(lib, dtype, algo, scale):
    """A negative scale turns the order of the scores round; 0 makes every weight equal."""
    _gpu()
    c = Case(dtype, 64, 1, 2, 1, 150, 150, 40, 3, seed=31)
    c.scale = scale
    c.check(algo)


@pytest.mark.gpu
@pytest.mark.parametrize("algo", [B.PSA_ALGO_SIMT, B.PSA_ALGO_AUTO])
def test_attention_repeats_bit_for_bit_and_in_graphs(lib, algo):
    """Two runs agree bit for bit; a captured forward and backward replay on new data."""
    torch = _gpu()
    c = Case("bf16", 64, 2, 4, 2, 700, 700, 100, 4, seed=9)
    o, lse = c.forward(algo)
    grads = c.backward(o, lse, algo)
    for _ in range(2):
        o2, lse2 = c.forward(algo)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert all(torch.equal(a, b) for a, b in zip(grads, c.backward(o, lse, algo)))
    ws = B.BwdWorkspace()
    q, k, v, do = (t.clone() for t in c.t)
    run = lambda: (lambda o, l: (o, l) + B.win_attn_bwd(q, k, v, o, l, do, c.scale, 100, 4, workspace=ws, algo=algo))(  # noqa: E731
        *B.win_attn_fwd(q, k, v, c.scale, 100, 4, algo=algo))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    other = Case("bf16", 64, 2, 4, 2, 700, 700, 100, 4, seed=10)
    for t, n in zip((q, k, v, do), other.t):
        t.copy_(n)
    g.replay()
    torch.cuda.synchronize()
    o, lse = other.forward(algo)
    want = (o, lse) + other.backward(o, lse, algo)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_without_rows_or_keys(lib, dtype):
    """No keys: O = 0, LSE = -inf, dQ = 0.  No rows: dK = dV = 0."""
    torch = _gpu()
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    t = lambda *n: torch.ones(n, dtype=dt, device="cuda")  # noqa: E731
    for Nq, Nk in ((130, 0), (0, 130), (0, 2000)):           # the last with far chunks of the sink rows
        q, k, v, do = t(2, 4, Nq, 64), t(2, 2, Nk, 64), t(2, 2, Nk, 64), t(2, 4, Nq, 64)
        o, lse = B.win_attn_fwd(q, k, v, 0.1, 40, 3)
        out = [torch.full_like(x, 7.0) for x in (q, k, v)]
        B.win_attn_bwd(q, k, v, o, lse, do, 0.1, 40, 3, dq=out[0], dk=out[1], dv=out[2])
        B.psa_attn_sync_status()
        assert (o == 0).all() and (lse == -INF).all() and all((x == 0).all() for x in out)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_on_two_streams_at_once(lib, dtype):
    """Forward and backward of two problems side by side, eager and as two graphs."""
    torch = _gpu()
    cases = [Case(dtype, d, 2, 4, 2, n, n, 100, 4, seed=d) for d, n in ((64, 900), (128, 500))]
    run = lambda c: (lambda o, l: (o, l) + c.backward(o, l))(*c.forward())  # noqa: E731
    want = [run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(cases[i]))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert all(torch.equal(a, b) for r in runs for a, b in zip(w, r))
    graphs, out = [torch.cuda.CUDAGraph() for _ in cases], []
    for g, c in zip(graphs, cases):
        with torch.cuda.graph(g):
            out.append(run(c))
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, o in zip(want, out) for a, b in zip(w, o))


@pytest.mark.gpu
def test_attention_on_another_stream(lib):
    torch = _gpu()
    c = Case("bf16", 128, 1, 4, 2, 300, 300, 64, 4, seed=12)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o, lse = c.forward()
        g = c.backward(o, lse)
    q, k, v, do = c.t
    for stream in (s, s.cuda_stream):                        # named in the call: a stream or its handle
        o3, lse3 = B.win_attn_fwd(q, k, v, c.scale, 64, 4, stream=stream)
        g3 = B.win_attn_bwd(q, k, v, o3, lse3, do, c.scale, 64, 4, stream=stream)
    s.synchronize()
    o2, lse2 = c.forward()
    assert torch.equal(o, o3) and all(torch.equal(a, b) for a, b in zip(g, g3))
    assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip(g, c.backward(o2, lse2)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_broadcast_inputs_and_far_strides(lib, dtype):
    """Keys shared by the batch through a zero stride, and heads more than 2^31 elements apart."""
    torch = _gpu()
    c = Case(dtype, 64, 2, 2, 1, 90, 90, 30, 2, seed=21)
    k1, v1 = c.t[1][:1].expand(2, -1, -1, -1), c.t[2][:1].expand(2, -1, -1, -1)
    q, _, _, do = c.t
    o, lse = B.win_attn_fwd(q, k1, v1, c.scale, 30, 2)
    o2, lse2 = B.win_attn_fwd(q, k1.contiguous(), v1.contiguous(), c.scale, 30, 2)
    # (the two may take different kernels: the same bounds, not the same bits)
    ref = W.batch_forward(c.q.astype(np.float64), *(np.repeat(x[:1], 2, 0).astype(np.float64) for x in (c.k, c.v)), c.scale,
                          30, 2, [90, 90], [90, 90], W.U[dtype])
    for got in ((o, lse), (o2, lse2)):
        _close(got[0], ref[0], ref[2], "O")
        _close(got[1], ref[1], ref[3], "LSE")
    far = torch.empty((1 << 31) + 90 * 64 * 2 + 16, dtype=q.dtype, device="cuda")
    views = []
    for i, t in enumerate(c.t[1:3]):
        v = far.as_strided((2, 1, 90, 64), (1 << 31, 64, 64, 1), i * 90 * 64)
        v.copy_(t)
        views.append(v)
    o3, lse3 = B.win_attn_fwd(q, *views, c.scale, 30, 2)
    o4, lse4 = B.win_attn_fwd(*c.t[:3], c.scale, 30, 2)
    g3 = B.win_attn_bwd(q, *views, o3, lse3, do, c.scale, 30, 2, dk=torch.empty_like(c.t[1]), dv=torch.empty_like(c.t[2]))
    g4 = B.win_attn_bwd(*c.t[:3], o4, lse4, do, c.scale, 30, 2)
    assert torch.equal(o3, o4) and all(torch.equal(a, b) for a, b in zip(g3, g4))


# ---------------------------------------------------------------- rotary positions
ROPES = [
    # d, sections, rot_dim, per_axis, interleaved
    (128, (64,), 128, False, False), (64, (8, 12, 12), 64, False, False), (32, (10, 6), 32, True, True),
    (16, (3, 5, 0), 16, True, False), (64, (5,), 10, False, False), (64, (4, 4), 16, False, True),
    (128, (16, 24, 24), 128, True, True), (32, (8,), 16, False, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["bnhd", "bhnd", "chan", "odd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rope", ROPES, ids=str)
def test_rope(lib, rope, dtype, layout):
    """Positions up to 2^31 - 1 and below 0.  A result is off by its rounding (u |y|), by
    the angle (2^-26 turns and the sine's own 2^-22) and by three fp32 operations on |x1| + |x2|."""
    torch = _gpu()
    d, sections, rot, per_axis, inter = rope
    rng = np.random.default_rng(d + rot)
    Bn, H, H2, N = 2, 3, 2, 37
    pos = rng.integers(-5000, 200000, size=(len(sections), Bn, N)).astype(np.int32)
    pos[:, 0, :4] = [0, 1, 2 ** 31 - 1, -2 ** 31]
    q, k = _draw(rng, (Bn, H, N, d), dtype), _draw(rng, (Bn, H2, N, d), dtype)
    plan = _plan(head_dim=d, sections=sections, rot_dim=rot, ladder=int(per_axis), interleaved=inter)
    tq, tk, tp = _dev(q, dtype, layout), _dev(k, dtype, layout), torch.from_numpy(pos).cuda()
    u = W.U[dtype]
    for inverse in (False, True):
        yq, yk = B.rope(plan, tq, tp, k=tk, inverse=inverse)
        for x, y in ((q, yq), (k, yk)):
            ref, mag = W.rotation(x, pos, sections, 10000.0, per_axis, inter, inverse)
            _close(y, ref, u * np.abs(ref) + mag * (2 * math.pi * 2.0 ** -26 + 2.0 ** -22 + 3 * W.U32), "rope")
            if rot < d:
                assert np.array_equal(_np(y)[..., rot:], x[..., rot:].astype(np.float64))
    assert torch.equal(B.rope(plan, tq, tp), B.rope(plan, tq, tp, k=tk)[0])
    for t in (tq, tk):                                       # in place
        want = B.rope(plan, t, tp)
        B.rope(plan, t, tp, out=t)
        assert torch.equal(t, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_on_packed_sections_and_shared_positions(lib, dtype):
    """The Q and K sections of a packed buffer rotate in place (a feature map's rows and
    columns as axes), positions shared by the batch; V sections stay as they were."""
    torch = _gpu()
    rng = np.random.default_rng(3)
    H, Wd, d, BH = 5, 7, 32, 3
    x = _draw(rng, (BH, 4, H * Wd, d), dtype)
    t = _dev(x, dtype, "bhnd")
    pos = np.stack([np.repeat(np.arange(H), Wd), np.tile(np.arange(Wd), H)]).astype(np.int32)
    plan = _plan(head_dim=d, sections=(8, 8), ladder=B.PSA_ROPE_PER_AXIS)
    B.rope(plan, t[:, :1], torch.from_numpy(pos).cuda(), k=t[:, 1:2], out=t[:, :1], out_k=t[:, 1:2])
    ref, mag = W.rotation(x[:, :2], np.repeat(pos[:, None], BH, 1), (8, 8), 10000.0, True, False, False)
    _close(t[:, :2], ref, W.U[dtype] * np.abs(ref) + mag * (2 * math.pi * 2.0 ** -26 + 2.0 ** -22 + 3 * W.U32), "rope")
    assert np.array_equal(_np(t[:, 2:]), x[:, 2:].astype(np.float64))


# ---------------------------------------------------------------- rolling cache
def _fill(rng, Bn, Hkv, cap, d, dtype):
    k, v = _draw(rng, (Bn, Hkv, cap, d), dtype), _draw(rng, (Bn, Hkv, cap, d), dtype)
    return k, v, _dev(k, dtype, "bhnd"), _dev(v, dtype, "bhnd")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["bnhd", "odd"])
@pytest.mark.parametrize("T,cap,sinks,start,n_new", [
    (1, 9, 2, [0, 1, 500], None), (5, 9, 2, [0, 7, 3], [5, 0, 2]), (40, 9, 2, [0, 7, 1], None), (40, 9, 0, [3, 9, 2], [40, 1, 77]),
    (12, 100, 4, [0, 2, 90], None), (6, 10, 3, [-1, 2 ** 31 - 4, 1], None), (700, 300, 4, [0, 31, 2], None),
])
def test_append(lib, dtype, layout, T, cap, sinks, start, n_new):
    """Every slot holds its newest position's key and value bit for bit, other slots what
    they held; a sequence with a start out of range is left as it was."""
    torch = _gpu()
    rng = np.random.default_rng(T + cap)
    Bn, Hkv, d = 3, 2, 32
    k, v, tk, tv = _fill(rng, Bn, Hkv, cap, d, dtype)
    kn, vn = _draw(rng, (Bn, Hkv, T, d), dtype), _draw(rng, (Bn, Hkv, T, d), dtype)
    c = B.WinCache(tk, tv, max(1, cap - sinks - 2), sinks)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c.append(_dev(kn, dtype, layout), _dev(vn, dtype, layout), i32(start), None if n_new is None else i32(n_new))
    for b in range(Bn):
        n = T if n_new is None else min(max(n_new[b], 0), T)
        if start[b] < 0 or start[b] + n > 2 ** 31 - 1:
            continue
        for t in range(n):
            s = W.slot(start[b] + t, cap, sinks)
            k[b, :, s], v[b, :, s] = kn[b, :, t], vn[b, :, t]
    assert np.array_equal(_np(tk), k.astype(np.float64)) and np.array_equal(_np(tv), v.astype(np.float64))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("layout", ["bnhd", "odd"])
def test_append_rotates_like_rope(lib, dtype, interleaved, layout):
    torch = _gpu()
    rng = np.random.default_rng(8)
    Bn, Hkv, T, d, cap = 2, 3, 50, 64, 64
    plan = _plan(head_dim=d, sections=(8, 12, 12), interleaved=interleaved)
    _, _, tk, tv = _fill(rng, Bn, Hkv, cap, d, dtype)
    kn, vn = (_dev(_draw(rng, (Bn, Hkv, T, d), dtype), dtype, layout) for _ in range(2))
    pos = torch.randint(0, 9999, (3, Bn, T), dtype=torch.int32, device="cuda")
    B.WinCache(tk, tv, 60, 4).append(kn, vn, torch.zeros(Bn, dtype=torch.int32, device="cuda"), plan=plan, pos=pos)
    assert torch.equal(tk[:, :, :T], B.rope(plan, kn, pos)) and torch.equal(tv[:, :, :T], vn)


def _decode_ref(q, k, v, lens, cap, window, sinks, scale, u):
    """q [B, Hq, d] over the cache's visible positions, gathered in order."""
    Bn, Hq, d = q.shape
    G = Hq // k.shape[1]
    o, bo, lse, bl = np.zeros(q.shape), np.zeros(q.shape), np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    for b in range(Bn):
        L = max(lens[b], 0)
        # sinks, then the window: as many gathered keys as the row sees
        pos = [p for p in list(range(min(sinks, max(L - window, 0)))) + list(range(max(L - window, 0), L))]
        at = [W.slot(p, cap, sinks) for p in pos]
        for h in range(Hq):
            if at:
                r = W.attention(q[b, h:h + 1], k[b, h // G, at], v[b, h // G, at], scale, len(at), 0, u)
                o[b, h], lse[b, h], bo[b, h], bl[b, h] = (x[0] for x in r)
    return o, lse, bo, bl


DECODES = [
    # Bn, Hq, Hkv, cap, window, sinks, lens
    (1, 1, 1, 1, 1, 0, [1]), (3, 2, 2, 9, 7, 2, [0, 1, 5]), (2, 4, 1, 9, 7, 2, [9, 1000]), (2, 7, 1, 40, 33, 4, [37, 12345]),
    (1, 8, 1, 300, 290, 4, [2000000000]), (4, 16, 2, 140, 128, 0, [-3, 64, 128, 129]), (1, 2, 2, 700, 600, 64, [650]),
    (2, 32, 1, 1100, 1024, 4, [1028, 5000]), (1, 24, 2, 5000, 4096, 17, [4999]), (16, 8, 8, 257, 200, 1, list(range(100, 260, 10))),
    (1, 65, 1, 130, 100, 2, [500]), (1, 4, 1, 40000, 33000, 4, [39000]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", DECODES, ids=lambda s: "-".join(str(x) for x in s[:6]))
def test_decode(lib, size, dtype, d):
    """Wrapped and unwrapped caches, empty sequences, garbage in every slot that is not visible."""
    torch = _gpu()
    Bn, Hq, Hkv, cap, window, sinks, lens = size
    rng = np.random.default_rng(cap + Hq)
    k, v, _, _ = _fill(rng, Bn, Hkv, 1, d, dtype)
    k, v = (round_storage(rng.normal(size=(Bn, Hkv, cap, d)), dtype) for _ in range(2))
    for b in range(Bn):
        L = max(lens[b], 0)
        seen = {W.slot(p, cap, sinks) for p in list(range(min(sinks, L))) + list(range(max(L - window, 0), L))}
        hidden = [s for s in range(cap) if s not in seen]
        k[b, :, hidden], v[b, :, hidden] = np.nan, np.inf
    q = _draw(rng, (Bn, Hq, d), dtype)
    tq = _dev(q[:, :, None], dtype, "bhnd")[:, :, 0]
    c = B.WinCache(_dev(k, dtype, "bhnd"), _dev(v, dtype, "bhnd"), window, sinks)
    lse = torch.empty((Bn, Hq), device="cuda")
    o = c.decode(tq, torch.tensor(lens, dtype=torch.int32, device="cuda"), 1 / math.sqrt(d), lse=lse)
    B.psa_attn_sync_status()
    ref = _decode_ref(q.astype(np.float64), k.astype(np.float64), v.astype(np.float64), lens, cap, window, sinks,
                      1 / math.sqrt(d), W.U[dtype])
    _close(o, ref[0], ref[2], "O")
    _close(lse, ref[1], ref[3], "LSE")
    assert torch.equal(o, c.decode(tq, torch.tensor(lens, dtype=torch.int32, device="cuda"), 1 / math.sqrt(d)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_layouts(lib, dtype):
    """Caches inside larger buffers: token-major [B, capacity, heads, d] and odd row strides;
    q and O as slices of a wider projection."""
    torch = _gpu()
    rng = np.random.default_rng(4)
    Bn, Hq, Hkv, cap, d, window, sinks, lens = 2, 6, 2, 90, 64, 70, 3, [55, 400]
    k, v = (_draw(rng, (Bn, Hkv, cap, d), dtype) for _ in range(2))
    q = _draw(rng, (Bn, Hq, d), dtype)
    tl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ref = _decode_ref(q.astype(np.float64), k.astype(np.float64), v.astype(np.float64), lens, cap, window, sinks, 0.125,
                      W.U[dtype])
    wide = torch.zeros((Bn, Hq + 2 * Hkv, d), dtype=_dev(q[:, :, None], dtype).dtype, device="cuda")
    wide[:, :Hq] = _dev(q[:, :, None], dtype)[:, :, 0]
    for layout in ("bhnd", "bnhd", "odd"):
        c = B.WinCache(_dev(k, dtype, layout), _dev(v, dtype, layout), window, sinks)
        out = torch.full((Bn, Hq + 1, d), 3.0, dtype=wide.dtype, device="cuda")
        c.decode(wide[:, :Hq], tl, 0.125, out=out[:, :Hq])
        _close(out[:, :Hq], ref[0], ref[2], layout)
        assert (out[:, Hq:] == 3.0).all()


@pytest.mark.gpu
def test_decode_and_append_past_32_bit_offsets(lib):
    """A cache of 2^32 elements: slots whose element offsets pass 32 bits."""
    torch = _gpu()
    cap, d = 1 << 25, 128
    k = torch.empty((1, 1, cap, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = B.WinCache(k, v, 200, 4)
    g = torch.Generator(device="cuda").manual_seed(1)
    new = [torch.randn((1, 1, 210, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    start = cap - 211
    i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    c.append(new[0][:, :, :4].contiguous(), new[1][:, :, :4].contiguous(), i32(0))
    c.append(*new, i32(start))
    q = torch.randn((1, 8, d), generator=g, device="cuda").to(torch.bfloat16)
    o = c.decode(q, i32(cap - 1), 0.1)
    small = B.WinCache(torch.cat([new[0][:, :, :4], new[0][:, :, 10:]], 2).contiguous(),
                       torch.cat([new[1][:, :, :4], new[1][:, :, 10:]], 2).contiguous(), 200, 4)
    assert torch.equal(k[0, 0, start:start + 210], new[0][0, 0])
    assert torch.equal(o, small.decode(q, i32(204), 0.1))


@pytest.mark.gpu
def test_decode_in_graphs_and_two_streams(lib):
    """Captured and replayed on new lengths; two caches at once on two streams."""
    torch = _gpu()
    rng = np.random.default_rng(6)
    caches = [B.WinCache(*(_dev(_draw(rng, (4, 2, 1100, 128), "bf16"), "bf16", "bhnd") for _ in range(2)), 1024, 4)
              for _ in range(2)]
    q = _dev(_draw(rng, (4, 8, 1, 128), "bf16"), "bf16", "bhnd")[:, :, 0]
    lens = torch.tensor([5, 900, 1028, 4000], dtype=torch.int32, device="cuda")
    want = [c.decode(q, lens, 0.09) for c in caches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in caches]
    got = [[], []]
    for _ in range(20):
        for i, (c, s) in enumerate(zip(caches, streams)):
            with torch.cuda.stream(s):
                got[i].append(c.decode(q, lens, 0.09))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = caches[0].decode(q, lens, 0.09)
    lens.copy_(torch.tensor([7, 1, 77, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, caches[0].decode(q, lens, 0.09))


@pytest.mark.gpu
def test_decode_in_a_graph_keeps_its_workspace(lib):
    """Calls with more query heads, whose workspace is larger, leave the captured one alone."""
    torch = _gpu()
    rng = np.random.default_rng(16)
    c = B.WinCache(*(_dev(_draw(rng, (1, 1, 9000, 64), "bf16"), "bf16", "bhnd") for _ in range(2)), 8192, 4)
    q = _dev(_draw(rng, (1, 48, 1, 64), "bf16"), "bf16", "bhnd")[:, :, 0]
    few = q[:, :4].contiguous()
    assert 0 < lib.psa_win_decode_workspace_bytes(c.c, 4) < lib.psa_win_decode_workspace_bytes(c.c, 48)
    lens = torch.tensor([9000], dtype=torch.int32, device="cuda")
    want = c.decode(few, lens, 0.1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = c.decode(few, lens, 0.1)
    c.decode(q, lens, 0.1)
    n = lib.psa_win_decode_workspace_bytes(c.c, 4)
    others = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for _ in range(8)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    assert all(bool((x == 77).all()) for x in others)


# ---------------------------------------------------------------- the operators together
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_training_step(lib, dtype):
    """Rotate, attend, and the gradients of both, against the oracle's chain in 64 bits.  The
    tolerances are the framework's own for a whole pass (the roundings between the operators
    add up): 1e-4 of the largest value for fp32, 2e-2 for bf16."""
    torch = _gpu()
    from gpu_helpers import TOL, rel_err
    rng = np.random.default_rng(31)
    Bn, Hq, Hkv, N, d, window, sinks, sections = 2, 4, 2, 150, 64, 40, 4, (8, 12, 12)
    x = [_draw(rng, (Bn, h, N, d), dtype) for h in (Hq, Hkv, Hkv, Hq)]
    pos = np.stack([np.stack([n // 100, n // 10 % 10, n % 10]) for n in (np.arange(N), np.arange(N) + 7)], 1).astype(np.int32)
    scale, plan = 0.125, _plan(head_dim=d, sections=sections)
    q, k, v, do = (_dev(t, dtype) for t in x)
    tp = torch.from_numpy(pos).cuda()
    rq, rk = B.rope(plan, q, tp, k=k)
    o, lse = B.win_attn_fwd(rq, rk, v, scale, window, sinks)
    drq, drk, dv = B.win_attn_bwd(rq, rk, v, o, lse, do, scale, window, sinks)
    dq, dk = B.rope(plan, drq, tp, k=drk, inverse=True)
    B.psa_attn_sync_status()
    f = [t.astype(np.float64) for t in x]
    turn = lambda t, inv: W.rotation(t, pos, sections, 10000.0, False, False, inv)[0]  # noqa: E731
    rq, rk = turn(f[0], False), turn(f[1], False)
    n = [N] * Bn
    ro, rl, _, _ = W.batch_forward(rq, rk, f[2], scale, window, sinks, n, n, 0.0)
    rdq, rdk, rdv = W.batch_gradient(rq, rk, f[2], ro, rl, f[3], scale, window, sinks, n, n, 0.0)[:3]
    for got, ref in ((o, ro), (dq, turn(rdq, True)), (dk, turn(rdk, True)), (dv, rdv)):
        assert rel_err(_np(got), ref) <= TOL[dtype]


@pytest.mark.gpu
def test_gradients_match_differences_of_the_forward(lib):
    """fp32: directional differences of the kernel's own forward.  The loss is a sum of n = B H N d
    terms, so its fp32 outputs' errors are far below h |<g, dir>| at h = 2^-6; the third-order
    term of the central difference is h^2 of the derivative, which 2e-3 covers."""
    torch = _gpu()
    c = Case("f32", 32, 1, 2, 1, 80, 80, 20, 2, seed=41)
    q, k, v, do = c.t
    o, lse = c.forward()
    grads = c.backward(o, lse)
    gen = torch.Generator(device="cuda").manual_seed(2)
    for i, g in enumerate(grads):
        step = torch.randn(g.shape, generator=gen, device="cuda")
        step = step / step.norm()
        loss = []
        for s in (2.0 ** -6, -2.0 ** -6):
            t = list(c.t[:3])
            t[i] = t[i] + s * step
            loss.append((B.win_attn_fwd(*t, c.scale, 20, 2)[0].double() * do.double()).sum())
        num = float((loss[0] - loss[1]) / 2.0 ** -5)
        assert abs(num - float((g.double() * step.double()).sum())) <= 2e-3 * float(g.double().norm())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("capacity", [68, 400])
def test_serving_follows_the_forward(lib, dtype, capacity):
    """A prompt and then token after token through the cache gives the rows of one forward pass
    over the whole sequence (within twice the bounds: both sides are compared with 64 bits)."""
    torch = _gpu()
    rng = np.random.default_rng(51)
    Bn, Hq, Hkv, N, d, window, sinks, prompt = 2, 4, 2, 300, 64, 60, 4, 283
    x = [_draw(rng, (Bn, h, N, d), dtype) for h in (Hq, Hkv, Hkv)]
    plan, scale = _plan(head_dim=d, sections=(32,)), 0.125
    q, k, v = (_dev(t, dtype) for t in x)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None]
    rq, rk = B.rope(plan, q, pos, k=k)
    o, lse = B.win_attn_fwd(rq, rk, v, scale, window, sinks)
    ref = W.batch_forward(_np(rq), _np(rk), x[2].astype(np.float64), scale, window, sinks, [N] * Bn, [N] * Bn, W.U[dtype])
    _close(o, ref[0], ref[2], "O")
    kc, vc = (torch.full((Bn, Hkv, capacity, d), float("nan"), dtype=q.dtype, device="cuda") for _ in range(2))
    c = B.WinCache(kc, vc, window, sinks)
    i32 = lambda n: torch.full((Bn,), n, dtype=torch.int32, device="cuda")  # noqa: E731
    c.append(k[:, :, :prompt], v[:, :, :prompt], i32(0), plan=plan, pos=pos[:, :prompt])
    for n in range(prompt, N):
        c.append(k[:, :, n:n + 1], v[:, :, n:n + 1], i32(n), plan=plan, pos=pos[:, n:n + 1])
        row = B.rope(plan, q[:, :, n:n + 1], pos[:, n:n + 1])
        got = c.decode(row[:, :, 0], i32(n + 1), scale)
        _close(got, ref[0][:, :, n], ref[2][:, :, n], f"row {n}")
