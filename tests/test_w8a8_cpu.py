"""int8 products and balance loss without a GPU: the oracle's functions against closed
forms and differences, and the refusals of the C entry points and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_ffn_15_b200 as moe
from mixture_experts_ffn_15_b200 import _abi
from mixture_experts_ffn_15_b200.build import build
from oracle import moe_oracle as O


def _lib():
    build()
    return _abi.load()


P = ctypes.c_void_p(4096)
BAD = ctypes.c_void_p(4104)   # not 16-byte aligned
OK, INV = _abi.MOE_OK, _abi.MOE_ERR_INVALID_ARG


# ------------------------------------------------------------------------- the oracle

def test_quantize_rows_closed_forms():
    x = np.array([[0.0, 0.0, 0.0, 0.0], [127.0, -127.0, 1.0, 0.5], [2.0, 1.0, -1.0, 0.0],
                  [1.0, np.inf, 0.0, 0.0], [np.nan, 1.0, 0.0, 0.0]])
    q, s = O.quantize_rows(x)
    assert q.tolist()[:3] == [[0, 0, 0, 0], [127, -127, 1, 0], [127, 64, -64, 0]]   # ties to even
    assert s[0] == 0 and s[1] == 1 and s[2] == np.float32(2) / np.float32(127)
    assert np.isnan(s[3]) and np.isnan(s[4]) and not q[3:].any()


def test_quantize_rows_is_nearest():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((20, 64)).astype(np.float32)
    q, s = O.quantize_rows(x)
    v = 127.0 * x.astype(np.float64) / np.abs(x).max(1, keepdims=True)
    assert np.all(np.abs(v - q) <= 0.5) and np.all(np.abs(q).max(1) == 127)
    # scaling a row by a power of two scales its scale alone
    q2, s2 = O.quantize_rows(x * 8)
    assert np.array_equal(q, q2) and np.array_equal(s * 8, s2)


def test_matmul_q8_is_the_dequantised_product():
    rng = np.random.default_rng(1)
    a = rng.integers(-127, 128, (5, 48))
    w = rng.integers(-127, 128, (32, 48))
    sa, sw = rng.uniform(0.1, 1, 5), rng.uniform(0.1, 1, 32)
    b = rng.standard_normal(32)
    want = (a * sa[:, None]) @ (w * sw[:, None]).T + b
    assert np.allclose(O.matmul_q8(a, sa, w, sw, b), want, rtol=1e-12)


@pytest.mark.parametrize("layout", ["interleaved", "chunked"])
def test_expert_ffn_w8a8_is_near_the_unrounded_ffn(layout):
    """Rounding either operand row to 8 bits moves a product by at most half a step of
    each element times the other operand's magnitudes; a loose consequence of it."""
    rng = np.random.default_rng(2)
    H, I, n = 64, 32, 7
    x = rng.standard_normal((n, H))
    q1, s1 = rng.integers(-127, 128, (2 * I, H)), rng.uniform(0.5, 1, 2 * I) / 127 / 8
    q2, s2 = rng.integers(-127, 128, (H, I)), rng.uniform(0.5, 1, H) / 127 / 6
    y = O.expert_ffn_w8a8(x, q1, s1, q2, s2, layout)
    ref = O.expert_ffn(x, q1 * s1[:, None], q2 * s2[:, None], layout)
    assert np.linalg.norm(y - ref) < 0.05 * np.linalg.norm(ref)
    other = "chunked" if layout == "interleaved" else "interleaved"
    assert np.linalg.norm(O.expert_ffn_w8a8(x, q1, s1, q2, s2, other) - ref) > 0.2 * np.linalg.norm(ref)


def test_balance_loss_closed_forms():
    T, E, k = 12, 6, 2
    idx = np.array([[t % E, (t + 1) % E] for t in range(T)])
    r = O.balance_loss(np.zeros((T, E)), idx, coef=0.5)
    assert r["loss"] == pytest.approx(0.5) and np.all(r["counts"] == T * k // E)
    assert np.allclose(r["probs"], 1 / E) and np.allclose(r["dlogits"], 0)
    # all tokens on one expert with certainty: E
    lg = np.full((T, E), -np.inf)
    lg[:, 3] = 0.0
    r = O.balance_loss(lg, np.full((T, 1), 3))
    assert r["loss"] == pytest.approx(E) and r["counts"][0, 3] == T
    # a masked batch is the batch without those tokens; halves as sequences average
    rng = np.random.default_rng(3)
    lg, idx = rng.standard_normal((T, E)), rng.integers(0, E, (T, k))
    keep = rng.random(T) < 0.6
    a, b = O.balance_loss(lg, idx, mask=keep), O.balance_loss(lg[keep], idx[keep])
    assert a["loss"] == pytest.approx(b["loss"]) and np.allclose(a["dlogits"][keep], b["dlogits"])
    assert not a["dlogits"][~keep].any()
    s = O.balance_loss(lg, idx, seq_offsets=[0, 5, 5, T])
    x, y = O.balance_loss(lg[:5], idx[:5]), O.balance_loss(lg[5:], idx[5:])
    assert s["loss"] == pytest.approx((x["loss"] + y["loss"]) / 3)


def test_balance_gradient_by_differences():
    rng = np.random.default_rng(4)
    T, E, k = 9, 5, 2
    lg, idx = rng.standard_normal((T, E)), rng.integers(0, E, (T, k))
    kw = dict(coef=0.3, mask=rng.random(T) < 0.8, seq_offsets=[0, 4, 8])
    g = O.balance_loss(lg, idx, **kw)["dlogits"]
    h = 1e-5
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(lg)
            d[t, e] = h
            num = (O.balance_loss(lg + d, idx, **kw)["loss"] - O.balance_loss(lg - d, idx, **kw)["loss"]) / (2 * h)
            # central differences: h^2 / 6 times a third derivative of order one
            assert abs(num - g[t, e]) < 1e-9


# ------------------------------------------------------------------------ refusals

def test_quantize_rows_refusals():
    lib = _lib()
    f = lambda x=P, rows=4, K=64, dt=1, q=P, s=P: lib.moe_quantize_rows(x, rows, K, dt, q, s, None)
    assert f(rows=0) == OK and f(rows=0, x=None) == OK
    assert f(rows=-1) == INV and f(K=0) == INV and f(K=12) == INV and f(dt=2) == INV
    assert f(x=None) == INV and f(q=None) == INV and f(s=None) == INV
    assert f(x=BAD) == INV and f(q=BAD) == INV and f(s=ctypes.c_void_p(4098)) == INV


def test_matmul_q8_refusals():
    lib = _lib()

    def f(a=P, sa=P, w=P, sw=P, b=None, off=P, rows=4, K=64, E=2, N=64, dt=1, out=P, err=None):
        return lib.moe_matmul_q8(a, sa, w, sw, b, off, rows, K, E, N, dt, out, err, None)
    assert f(rows=0) == OK
    assert f(rows=-1) == INV and f(E=0) == INV and f(E=257) == INV and f(dt=3) == INV
    assert f(K=24) == INV and f(K=0) == INV and f(K=65552) == INV     # 16-byte rows, int32 sums
    assert f(N=48) == INV and f(N=0) == INV
    assert f(off=None) == INV                                         # no offsets: one expert
    for n in ("a", "sa", "w", "sw", "out"):
        assert f(**{n: None}) == INV
    for n in ("a", "w", "out"):
        assert f(**{n: BAD}) == INV
    odd = ctypes.c_void_p(4097)
    for n in ("sa", "sw", "b", "off", "err"):
        assert f(**{n: odd}) == INV


def test_expert_ffn_w8a8_refusals():
    lib = _lib()

    def f(x=P, off=P, w1=P, s1=P, w2=P, s2=P, b1=None, b2=None, rows=4, H=64, E=2, I=32,
          act=_abi.STANDARD_SWIGLU, layout=0, y=P, ws=P, nb=1 << 40):
        return lib.moe_expert_ffn_w8a8(x, off, w1, s1, w2, s2, b1, b2, rows, H, E, I, act, layout, y, ws, nb, None)
    assert f(rows=0) == OK
    assert f(rows=-1) == INV and f(H=48) == INV and f(I=16) == INV and f(E=0) == INV and f(E=300) == INV
    assert f(layout=2) == INV and f(act=_abi.MoeSwiglu(1.0, 0.0, -1.0)) == INV
    need = lib.moe_expert_ffn_w8a8_workspace_size(4, 64, 2, 32)
    assert need > 0 and f(nb=need - 1) == INV
    assert lib.moe_expert_ffn_w8a8_workspace_size(4, 48, 2, 32) == 0
    for n in ("x", "off", "w1", "s1", "w2", "s2", "y", "ws"):
        assert f(**{n: None}) == INV
    for n in ("x", "w1", "w2", "y", "ws"):
        assert f(**{n: BAD}) == INV
    assert f(b1=ctypes.c_void_p(4097)) == INV


def test_more_than_2_30_rows_are_refused():
    """Row counts whose tiles and launch sizes would pass 32 bits."""
    lib, many = _lib(), (1 << 30) + 1
    assert lib.moe_quantize_rows(P, many, 64, 1, P, P, None) == INV
    assert lib.moe_matmul_q8(P, P, P, P, None, P, many, 64, 2, 64, 1, P, None, None) == INV
    assert lib.moe_expert_ffn_w8a8_workspace_size(many, 64, 2, 32) == 0
    assert lib.moe_expert_ffn_w8a8_workspace_size(1 << 30, 64, 2, 32) > (1 << 30) * 64
    assert lib.moe_expert_ffn_w8a8(P, P, P, P, P, P, None, None, many, 64, 2, 32, _abi.STANDARD_SWIGLU, 0, P, P,
                                   (1 << 63) - 1, None) == INV


def test_forward_w8a8_refusals():
    lib = _lib()

    def f(x=P, nw=None, eps=1e-6, rw=P, rb=None, w1=P, s1=P, w2=P, s2=P, T=4, H=64, E=8, k=2, I=32,
          act=_abi.STANDARD_SWIGLU, layout=0, out=P, ws=P, nb=1 << 40):
        return lib.moe_forward_w8a8(x, nw, eps, rw, rb, w1, s1, w2, s2, None, None, T, H, E, k, I, 1, act, layout,
                                    out, ws, nb, None)
    assert f(T=0) == OK
    assert f(T=-1) == INV and f(k=9) == INV and f(H=40) == INV and f(I=16) == INV and f(E=257) == INV
    assert f(nw=P, eps=-1.0) == INV and f(nw=BAD) == INV
    need = lib.moe_w8a8_workspace_size(4, 64, 8, 2, 32)
    assert need > 0 and f(nb=need - 1) == INV and lib.moe_w8a8_workspace_size(4, 64, 8, 9, 32) == 0
    for n in ("x", "rw", "w1", "s1", "w2", "s2", "out", "ws"):
        assert f(**{n: None}) == INV


def test_balance_refusals():
    lib = _lib()

    def f(lg=P, idx=P, mask=None, seq=None, T=8, E=4, k=2, S=1, coef=1.0, out=P, err=None, ws=P, nb=1 << 40):
        return lib.moe_balance_loss(lg, idx, mask, seq, T, E, k, S, coef, out, P, P, P, err, ws, nb, None)

    def g(lg=P, seq=None, cnt=P, n=P, T=8, E=4, k=2, S=1, coef=1.0, gl=None, d=P):
        return lib.moe_balance_loss_backward(lg, None, seq, cnt, n, T, E, k, S, coef, gl, d, None)
    for c in (f, g):
        assert c(T=-1) == INV and c(E=0) == INV and c(E=257) == INV and c(k=0) == INV and c(k=5) == INV
        assert c(S=0) == INV and c(S=2) == INV and c(S=70000, seq=P) == INV and c(coef=float("nan")) == INV
        assert c(lg=None) == INV and c(lg=BAD) == INV and c(T=1 << 30, k=2) == INV
    assert f(idx=None) == INV and f(out=None) == INV and f(ws=BAD) == INV
    need = lib.moe_balance_loss_workspace_size(8, 4, 1)
    assert need > 0 and f(nb=need - 1) == INV
    assert lib.moe_balance_loss_workspace_size(8, 4, 0) == 0
    assert g(T=0) == OK and g(cnt=None) == INV and g(n=None) == INV and g(d=BAD) == INV
    assert g(gl=ctypes.c_void_p(4098)) == INV


def test_binding_refuses_cpu_tensors_types_and_shapes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        moe.quantize_rows(x)
    with pytest.raises(ValueError, match="CUDA"):
        moe.matmul_q8(q, s, q, s)
    with pytest.raises(ValueError, match="CUDA"):
        moe.expert_ffn_w8a8(x, s, q, s, q, s)
    with pytest.raises(ValueError, match="CUDA"):
        moe.forward_w8a8(x, x, q[None], s, q[None], s, 1)
    with pytest.raises(ValueError, match="CUDA"):
        moe.balance_loss(s[:, None], s[:, None].int())
    with pytest.raises(ValueError, match="CUDA"):
        moe.balance_loss_backward(s[:, None], 1, s, s)


def test_workspaces_grow_and_are_whole_blocks():
    lib = _lib()
    a = lib.moe_expert_ffn_w8a8_workspace_size(100, 256, 8, 128)
    assert a % 256 == 0 and a >= 100 * (256 + 4 + 128 + 4)
    assert lib.moe_expert_ffn_w8a8_workspace_size(101, 256, 8, 128) >= a
    assert lib.moe_w8a8_workspace_size(50, 256, 8, 2, 128) > a
    assert lib.moe_balance_loss_workspace_size(0, 8, 3) > 0
