"""The window attention family where it could go wrong unseen: workspaces used again with other
inputs, values and positions at the ends of their ranges, many work items per block.  A
result that is NaN where the reference is finite fails here."""
import math

import numpy as np
import pytest

import test_window as T
import window_oracle as W
from self_attention_backward_gb300 import binding as B

lib = T.lib


def close(got, ref, bound, what):
    """test_window's comparison, where its `err > bound` lets a NaN pass."""
    got = T._np(got) if not isinstance(got, np.ndarray) else got
    fin = np.isfinite(ref)
    assert np.array_equal(got[~fin], ref[~fin]), what
    over = ~(np.abs(got[fin] - ref[fin]) <= bound[fin] + 1e-30)
    assert not over.any(), (what, int(over.sum()), got[fin][over][:4], ref[fin][over][:4])


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    monkeypatch.setattr(T, "_close", close)


# ---------------------------------------------------------------- no NaN for a number
def test_close_sees_a_nan():
    ref, bound = np.array([1.0, -np.inf]), np.array([0.5, 0.0])
    close(np.array([1.25, -np.inf]), ref, bound, "")
    for bad in ([np.nan, -np.inf], [np.inf, -np.inf], [1.0, np.nan], [1.6, -np.inf]):
        with pytest.raises(AssertionError):
            close(np.array(bad), ref, bound, "")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("dtype,algo", T.ALGOS)
@pytest.mark.parametrize("size", T.SIZES, ids=lambda s: "-".join(str(x) for x in s[:7]))
def test_attention_is_finite(lib, size, dtype, algo, d):
    T.test_attention(lib, size, dtype, algo, d)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,algo", T.ALGOS)
def test_attention_is_finite_at_the_edges(lib, dtype, algo):
    for d in (16, 64, 128):
        T.test_attention_padding_is_never_read(lib, dtype, algo, d)
    T.test_attention_large_scores(lib, dtype, algo)
    for scale in (-0.2, 0.0, 1e-3):
        T.test_attention_scales(lib, dtype, algo, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layouts_are_finite(lib, dtype):
    for layout in ("bhnd", "chan", "odd"):
        T.test_attention_layouts(lib, dtype, layout)
    T.test_attention_broadcast_inputs_and_far_strides(lib, dtype)
    T.test_decode_layouts(lib, dtype)
    for capacity in (68, 400):
        T.test_serving_follows_the_forward(lib, dtype, capacity)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["bnhd", "chan", "odd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_is_finite(lib, dtype, layout):
    for rope in T.ROPES:
        T.test_rope(lib, rope, dtype, layout)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", T.DECODES, ids=lambda s: "-".join(str(x) for x in s[:6]))
def test_decode_is_finite(lib, size, dtype, d):
    T.test_decode(lib, size, dtype, d)


# ---------------------------------------------------------------- the build
def test_library_builds_without_python_headers(lib, monkeypatch, tmp_path):
    """The C library does not need what the Python side needs; a compiler's error is one all the same."""
    from self_attention_backward_gb300 import build as M
    monkeypatch.setattr(M, "BIND", str(tmp_path / "bind.so"))
    paths, which = M.sysconfig.get_paths(), M.shutil.which
    with monkeypatch.context() as m:
        m.setattr(M.sysconfig, "get_paths", lambda: dict(paths, include=str(tmp_path)))
        with pytest.warns(UserWarning, match="Python.h"):
            assert M.build() == M.LIB
    with monkeypatch.context() as m:
        m.setattr(M.shutil, "which", lambda n: None if n == "gcc" else which(n))
        with pytest.warns(UserWarning, match="gcc"):
            assert M.build() == M.LIB
    assert not (tmp_path / "bind.so").exists()
    (tmp_path / "Python.h").write_text("#error no\n")
    monkeypatch.setattr(M.sysconfig, "get_paths", lambda: dict(paths, include=str(tmp_path)))
    with pytest.raises(M.subprocess.CalledProcessError):
        M.build()


def test_binding_module_is_this_interpreters(lib):
    """Another Python's module has another name."""
    import sysconfig
    from self_attention_backward_gb300 import build as M
    assert M.BIND == B.BIND_PATH and M.BIND.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


# ---------------------------------------------------------------- how often a bf16 result is rounded
@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("algo,roundings", [(B.PSA_ALGO_TC, 2), (B.PSA_ALGO_SIMT, 1)])
def test_bf16_results_are_rounded_as_often_as_said(lib, algo, roundings, d):
    """A rounding to bf16 takes r = 0.00166 of the norm (normal or exponential values); k of them
    that are independent take sqrt(k) r.  The tensor cores' O, dQ, dK and dV are rounded twice: P or dS
    for the product, dS from fp32 P, then the result; the warp-level products' once.  One more would
    pass the limit half a rounding higher."""
    T._gpu()
    c = T.Case("bf16", d, 2, 4, 2, 700, 700, 700, 0, seed=101)
    o, lse = c.forward(algo)
    f = lambda x: x.astype(np.float64)  # noqa: E731
    n = [700, 700]
    ro = W.batch_forward(f(c.q), f(c.k), f(c.v), c.scale, 700, 0, n, n, 0.0)[0]
    ref = W.batch_gradient(f(c.q), f(c.k), f(c.v), T._np(o), T._np(lse), f(c.do), c.scale, 700, 0, n, n, 0.0)[:3]
    limit = 0.00166 * math.sqrt(roundings + 0.5)
    for name, g, r in zip(("O", "dQ", "dK", "dV"), (o, *c.backward(o, lse, algo)), (ro, *ref)):
        assert np.linalg.norm(T._np(g) - r) <= limit * np.linalg.norm(r), name


# ---------------------------------------------------------------- more work items than SMs
MANY = [
    # Bn, Hq, Hkv, Nq, Nk, window, sinks, q_lens, kv_lens.  On 152 SMs, items of the forward, dK/dV, dQ:
    # 192, 192, 384; an empty sequence and one without rows that see anything in between
    (8, 8, 4, 700, 700, 130, 4, [700, 0, 513, 1, 700, 128, 640, 333], [700, 0, 600, 5, 650, 700, 640, 0]),
    # 320, 200, 600; three query heads per key head; more rows than keys
    (8, 15, 5, 600, 610, 70, 0, [600, 600, 30, 600, 599, 0, 257, 600], [610, 1, 610, 500, 600, 77, 256, 128]),
    # 192, 240 (far chunks of the sink rows among them), 384
    (4, 8, 4, 1500, 1500, 60, 5, [1500, 1, 1100, 1500], [1500, 1500, 1300, 700]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("size", MANY, ids=lambda s: "-".join(str(x) for x in s[:7]))
def test_attention_of_many_items(lib, size, d):
    """Every persistent block takes several items: stages, barriers and TMEM carried from one to
    the next, items without work among them, anything in the padding."""
    T._gpu()
    if size[3] >= 1000 and d not in (32, 128):
        pytest.skip("the longest sequences at two head sizes")
    c = T.Case("bf16", d, *size, seed=80 + d, garbage=True)
    c.check(B.PSA_ALGO_TC)


@pytest.mark.gpu
def test_attention_of_many_items_repeats(lib):
    """The same bits with four and more items a block, alone and beside another stream's work."""
    torch = T._gpu()
    c = T.Case("bf16", 64, 8, 16, 8, 900, 900, 200, 3, seed=91)
    o, lse = c.forward()
    want = (o, lse, *c.backward(o, lse))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        with torch.cuda.stream(side):
            a = c.forward()
            a = (*a, *c.backward(*a))
        b = c.forward()
        b = (*b, *c.backward(*b))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g in (a, b) for x, y in zip(want, g))
    B.psa_attn_sync_status()


CLUSTERS = [
    # a cluster of 8 shares a dK/dV item: 4 items of 32 tiles; with far chunks and sink rows; ragged
    (1, 8, 1, 400, 400, 400, 0, None, None),
    (1, 8, 1, 1500, 1500, 60, 4, None, None),
    (2, 16, 1, 300, 420, 90, 130, [300, 111], [420, 200]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("size", CLUSTERS, ids=lambda s: "-".join(str(x) for x in s[:7]))
def test_backward_shared_by_clusters(lib, size, d):
    T._gpu()
    T.Case("bf16", d, *size, seed=95 + d, garbage=True).check(B.PSA_ALGO_TC)


MANY_ROWS = [
    # dtype, d, H, H2, N, sections, rot_dim, interleaved: more than 608 groups, the last one partial
    ("bf16", 64, 5, 3, 2701, (8, 12, 12), 64, False),        # 8 tokens a group
    ("bf16", 128, 3, 2, 2701, (24, 8), 64, True),            # features past the rotated ones
    ("f32", 32, 7, 2, 2101, (16,), 32, False),
    ("f32", 128, 17, 2, 611, (40, 24), 128, True),           # heads in two parts, the second smaller
]


@pytest.mark.gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("rope", MANY_ROWS, ids=str)
def test_rope_of_many_rows(lib, rope, inverse):
    """Blocks that go through several groups of several tokens.  Bounds as in test_rope."""
    torch = T._gpu()
    dtype, d, H, H2, N, sections, rot, inter = rope
    rng = np.random.default_rng(N + d)
    pos = rng.integers(0, 200000, size=(len(sections), 2, N)).astype(np.int32)
    q, k = T._draw(rng, (2, H, N, d), dtype), T._draw(rng, (2, H2, N, d), dtype)
    plan = T._plan(head_dim=d, sections=sections, rot_dim=rot, interleaved=inter)
    tq, tk, tp = T._dev(q, dtype), T._dev(k, dtype), torch.from_numpy(pos).cuda()
    yq, yk = B.rope(plan, tq, tp, k=tk, inverse=inverse)
    for x, y in ((q, yq), (k, yk)):
        ref, mag = W.rotation(x, pos, sections, 10000.0, False, inter, inverse)
        close(y, ref, W.U[dtype] * np.abs(ref) + mag * (2 * math.pi * 2.0 ** -26 + 2.0 ** -22 + 3 * W.U32), "rope")
    B.rope(plan, tq, tp, k=tk, inverse=inverse, out=tq, out_k=tk)
    assert torch.equal(tq, yq) and torch.equal(tk, yk)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,Hkv,T_", [("bf16", 64, 4, 2000), ("f32", 128, 3, 1100), ("bf16", 128, 17, 700)])
def test_append_of_many_rows(lib, dtype, d, Hkv, T_):
    """Several groups per block with a rotation: keys as rope leaves them, values as they are, in
    the newest position's slot; other slots untouched."""
    torch = T._gpu()
    rng = np.random.default_rng(d)
    Bn, sinks, cap = 3, 5, T_ - 100
    plan = T._plan(head_dim=d, sections=(d // 4, d // 4))
    _, _, tk, tv = T._fill(rng, Bn, Hkv, cap, d, dtype)
    want = [tk.clone(), tv.clone()]
    kn, vn = (T._dev(T._draw(rng, (Bn, Hkv, T_, d), dtype), dtype) for _ in range(2))
    pos = torch.randint(0, 9999, (2, Bn, T_), dtype=torch.int32, device="cuda")
    start, n_new = [0, 7777, 3], [T_, T_, T_ - 333]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    B.WinCache(tk, tv, cap - sinks, sinks).append(kn, vn, i32(start), n_new=i32(n_new), plan=plan, pos=pos)
    rk = B.rope(plan, kn, pos)
    for b in range(Bn):
        holds = {W.slot(start[b] + t, cap, sinks): t for t in range(n_new[b])}
        slots, rows = list(holds), list(holds.values())
        want[0][b][:, slots] = rk[b][:, rows]
        want[1][b][:, slots] = vn[b][:, rows]
    assert torch.equal(tk, want[0]) and torch.equal(tv, want[1])


# ---------------------------------------------------------------- the ends of ranges
def test_cache_refuses_slots_past_2_30(lib):
    """A ring's first slot plus a visible position has to stay in 32 bits.  (The pointers are never
    used: the calls fail their checks first.)"""
    v = T._view()
    big = lambda cap: T._cache(kv_heads=1, capacity=cap, head_dim=16, window=1 << 20, batch_stride=1 << 36,  # noqa: E731
                               head_stride=1 << 35, slot_stride=16)
    for cap in (2 ** 30 + 1, 2 ** 31 - 1):
        assert lib.psa_win_decode(big(cap), v, v, None, 4, T.FAKE, 0.5, T.FAKE, 1 << 40, None) == B.PSA_ERR_UNSUPPORTED
        assert lib.psa_win_cache_append(big(cap), v, v, 8, T.FAKE, None, None, None, 0, 0, None) == B.PSA_ERR_UNSUPPORTED
        assert lib.psa_win_decode_workspace_bytes(big(cap), 4) == 0
    assert lib.psa_win_decode_workspace_bytes(big(2 ** 30), 4) > 0
    one = T._cache(kv_heads=1, head_dim=16, batch_stride=128, head_stride=128, slot_stride=16)
    n = B.psa_attn_view(T.FAKE, 0, 0, 16, 1)
    assert lib.psa_win_cache_append(one, n, n, 2 ** 30 + 1, T.FAKE, None, None, None, 0, 0, None) == B.PSA_ERR_UNSUPPORTED


def test_rope_refuses_rows_past_2_30(lib):
    v = B.psa_attn_view(T.FAKE, 0, 0, 16, 1)
    call = lambda n: lib.psa_rope(T._plan(head_dim=16, sections=(8,)).c, v, v, 1, None, None, 0, 1, n, None, 0, 0, 0,  # noqa: E731
                                  B.PSA_BF16, None)
    assert call(2 ** 31 - 1) == B.PSA_ERR_UNSUPPORTED
    assert call(2 ** 30 + 1) == B.PSA_ERR_UNSUPPORTED
    assert call(2 ** 30) == B.PSA_ERR_ARG                    # the size passes, the missing positions do not


def test_sizes_past_32_bits_are_not_cut_off(lib):
    """2^32 + 4 is not 4."""
    torch = pytest.importorskip("torch")
    k, big = torch.zeros((1, 1, 16, 16)), 2 ** 32
    assert B.WinCache(k, k.clone(), 4, 1).c.window == 4
    assert list(T._plan(sections=(32 / 4, 8)).c.axis[:16]) == [0] * 8 + [1] * 8
    for call in (lambda: B.WinCache(k, k.clone(), big + 4, 1), lambda: B.WinCache(k, k.clone(), 4, big + 1),
                 lambda: B.WinCache(k, k.clone(), 4, -big), lambda: B.WinCache(k.expand(1, 1, 16, 16), k, 4.5, 1),
                 lambda: B.WinCache(*[torch.zeros((1, 1, 1, 16)).expand(1, 1, big + 16, 16)] * 2, 4, 1),
                 lambda: T._plan(head_dim=big + 32), lambda: T._plan(rot_dim=big + 32),
                 lambda: T._plan(sections=(big + 8, 8)), lambda: T._plan(ladder=big)):
        with pytest.raises((ValueError, TypeError)):
            call()


@pytest.mark.parametrize("theta", [10000.0, 500.0, 1e6, 1.0 + 2.0 ** -40, 1.5, 1e300])
def test_plan_fractions_are_rounded_exactly(lib, theta):
    """Every turn fraction is the nearest multiple of 2^-64, or the next where the two are as good as
    equally near (2^-10 of a unit): decimals of 60 digits."""
    from decimal import Decimal as D, localcontext
    with localcontext() as ctx:
        ctx.prec = 60
        two_pi = 2 * D("3.14159265358979323846264338327950288419716939937510582097494")
        ln = D(theta).ln()
        for sections, per_axis in (((64,), 0), ((16, 24, 24), 0), ((16, 24, 24), 1), ((1, 63), 1), ((0, 7, 57), 1)):
            p = T._plan(head_dim=128, sections=sections, theta=theta, ladder=per_axis).c
            e = [D(k) / s for s in sections for k in range(s)] if per_axis else [D(i) / 64 for i in range(64)]
            for i, x in enumerate(e):
                assert abs(p.turn[i] - (-ln * x).exp() / two_pi * 2 ** 64) <= D(0.5) + D(2) ** -10, (sections, i)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["bnhd", "odd"])
def test_append_up_to_the_last_position(lib, dtype, layout):
    """Positions up to 2^31 - 1 are written; one more skips the sequence."""
    torch = T._gpu()
    rng = np.random.default_rng(77)
    Bn, Hkv, d, Tn, cap, sinks, last = 4, 2, 32, 6, 11, 3, 2 ** 31 - 1
    k, v, tk, tv = T._fill(rng, Bn, Hkv, cap, d, dtype)
    kn, vn = T._draw(rng, (Bn, Hkv, Tn, d), dtype), T._draw(rng, (Bn, Hkv, Tn, d), dtype)
    start, n_new = [last - 5, last - 4, last, last], [6, 6, 1, 0]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    B.WinCache(tk, tv, 8, sinks).append(T._dev(kn, dtype, layout), T._dev(vn, dtype, layout), i32(start), i32(n_new))
    for b, rows in ((0, range(6)), (2, range(1))):
        for t in rows:
            s = W.slot(start[b] + t, cap, sinks)
            k[b, :, s], v[b, :, s] = kn[b, :, t], vn[b, :, t]
    assert np.array_equal(T._np(tk), k.astype(np.float64)) and np.array_equal(T._np(tv), v.astype(np.float64))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64])
def test_attention_of_the_largest_numbers(lib, d):
    """fp32 values up to the largest finite one, where their products stay finite: q's against keys
    of some 2^-126, v's and q's (in dK) alone in their features; dO is 0 where v is large."""
    T._gpu()
    c = T.Case("f32", d, 1, 2, 1, 70, 70, 20, 2, seed=71)
    big = np.finfo(np.float32).max
    c.q[:, :, :, 3], c.k[:, :, :, 3] = 0.0, np.ldexp(1 + np.arange(70) % 32 / 32, -126)
    c.q[0, :, 40, 3], c.q[0, 1, 3, 3] = big, -float.fromhex("0x1.ffep127")
    c.v[:, :, :, 5:7] = c.do[:, :, :, 5:7] = 0.0
    c.v[0, 0, 33, 5], c.v[0, 0, 1, 6] = big, -np.nextafter(big, np.float32(0))
    c.t = [T._dev(x.astype(np.float32), "f32") for x in (c.q, c.k, c.v, c.do)]
    o, lse = c.forward()
    f = lambda *x: [a.astype(np.float64) for a in x]  # noqa: E731
    ref = W.batch_forward(*f(c.q, c.k, c.v), c.scale, 20, 2, [70], [70], W.U["f32"])
    close(o, ref[0], ref[2], "O")
    close(lse, ref[1], ref[3], "LSE")
    got = [T._np(g) for g in c.backward(o, lse)]
    ref = W.batch_gradient(*f(c.q, c.k, c.v), T._np(o), T._np(lse), *f(c.do), c.scale, 20, 2, [70], [70], W.U["f32"])
    # dK = scale (dS^T Q): a partial sum of the bracket may pass the largest fp32 number, and be
    # infinite, where the absolute values of its terms add up to more (4.2e38 at d=32)
    past, terms = ~np.isfinite(got[1]), np.zeros(got[1].shape)
    for h in range(2):
        q, k, v, do = f(c.q[0, h], c.k[0, 0], c.v[0, 0], c.do[0, h])
        s = np.where(W.visible(70, 70, 20, 2), q @ k.T * c.scale, -np.inf)
        ds = np.exp(s - T._np(lse)[0, h][:, None]) * (do @ v.T - (do * T._np(o)[0, h]).sum(-1, keepdims=True))
        terms[0, 0] += np.abs(ds).T @ np.abs(q)
    assert past.sum() < 10 and (terms[past] > big).all() and not np.isnan(got[1]).any()
    got[1][past] = ref[1][past]
    for name, g, r, bound in zip(("dQ", "dK", "dV"), got, ref[:3], ref[3:]):
        close(g, r, bound, name)
    assert o.abs().max() > 1e36 and np.sort(np.abs(got[1]), None)[-15] > 1e36


def test_too_many_items_are_refused_before_any_launch(lib):
    """(Without a device a launch answers with a CUDA error.)"""
    n = 2 ** 10 + 1
    for kw, algo in ((dict(), B.PSA_ALGO_TC), (dict(Nk=33), B.PSA_ALGO_SIMT)):
        s = T._shape(B=2 ** 20, q_heads=n, kv_heads=n, Nq=1, head_dim=16, **dict(dict(Nk=1), **kw))
        v = B.psa_attn_view(T.FAKE, 16 * n * s.Nk, 16 * s.Nk, 16, 1)
        call = lambda: lib.psa_win_attn_bwd(s, v, v, v, v, T.FAKE, v, v, v, v, None, None, T.FAKE, 1 << 60, algo, None)  # noqa: E731
        assert call() == B.PSA_ERR_UNSUPPORTED and "too large" in B.psa_attn_last_error()
        if algo == B.PSA_ALGO_TC:
            assert lib.psa_win_attn_fwd(s, v, v, v, v, T.FAKE, None, None, algo, None) == B.PSA_ERR_UNSUPPORTED


# ---------------------------------------------------------------- streams
def test_stream_of_another_device_is_refused(lib):
    """(It was dropped: the call ran on the current stream of the tensors' device.)"""
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    there = SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    q = SimpleNamespace(device=torch.device("cuda:0"))
    cache = B.WinCache(torch.zeros((1, 1, 16, 16)), torch.zeros((1, 1, 16, 16)), 4, 1)
    cache.device = q.device
    for call in (lambda: B.win_attn_fwd(q, q, q, 1.0, 4, 0, stream=there), lambda: B.rope(T._plan(), q, None, stream=there),
                 lambda: B.win_attn_bwd(q, q, q, q, None, q, 1.0, 4, 0, stream=there),
                 lambda: cache.append(q, q, None, stream=there), lambda: cache.decode(q, None, 1.0, stream=there)):
        with pytest.raises(ValueError, match="stream is of cuda:1"):
            call()


@pytest.mark.gpu
def test_a_cache_may_go_while_another_stream_decodes(lib):
    """The workspace of a call belongs to the call's stream: memory that a cache which is gone gives
    back is not handed out on another one before the call has ended."""
    torch = T._gpu()
    rng = np.random.default_rng(17)
    k, v = (T._dev(T._draw(rng, (1, 1, 9000, 64), "bf16"), "bf16", "bhnd") for _ in range(2))
    q = T._dev(T._draw(rng, (1, 8, 1, 64), "bf16"), "bf16", "bhnd")[:, :, 0]
    lens = torch.tensor([9000], dtype=torch.int32, device="cuda")
    c = B.WinCache(k, v, 8192, 4)
    n = lib.psa_win_decode_workspace_bytes(c.c, 8)
    assert n > 0
    want = c.decode(q, lens, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                        # some 10 ms
        got = c.decode(q, lens, 0.1)
    del c
    others = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(bool((x == 77).all()) for x in others)


# ---------------------------------------------------------------- one call's data in another


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["bnhd", "odd"])
@pytest.mark.parametrize("dtype,algo", T.ALGOS)
def test_backward_uses_this_calls_statistics(lib, dtype, algo, layout):
    """Calls that share a workspace in turn on different inputs give what each gives with one of
    its own, bit for bit: row statistics, inputs and outputs lie at the same addresses every time."""
    torch = T._gpu()
    *cases, spare = [T.Case(dtype, 32, 2, 4, 2, 700, 700, 150, 2, seed=60 + i, layout=layout) for i in range(3)]
    fwd = [c.forward(algo) for c in cases]
    want = [c.backward(*f, algo=algo) for c, f in zip(cases, fwd)]
    torch.cuda.synchronize()
    ins = (*spare.t, *spare.forward(algo))
    ws = B.BwdWorkspace()
    got = []
    for n in range(40):
        for to, t in zip(ins, (*cases[n % 2].t, *fwd[n % 2])):
            to.copy_(t)
        q, k, v, do, o, lse = ins
        got.append(B.win_attn_bwd(q, k, v, o, lse, do, cases[0].scale, 150, 2, workspace=ws, algo=algo))
    B.psa_attn_sync_status()
    for n, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(want[n % 2], g)), n
