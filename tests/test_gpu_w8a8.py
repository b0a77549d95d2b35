"""int8 rows, int8 x int8 products, the expert FFN and the layer on them, on the GPU.

Whole numbers are compared bit for bit; products and the FFN against float64 within the
bounds of w8a8_util (derived there)."""
import ctypes

import numpy as np
import pytest
import torch

import mixture_experts_ffn_15_b200 as moe
from mixture_experts_ffn_15_b200 import _abi
from oracle import moe_oracle as O
from parity_util import assert_close, device_inputs, from_dev, match_routing
from synth import Workload, make_inputs, make_q8_experts
from w8a8_util import (TORCH, check, ffn_with_bound, product_bound, rounded, split, weights)

pytestmark = pytest.mark.gpu

STD, OSS = (1.0, 0.0, float("inf")), (1.702, 1.0, 7.0)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# --------------------------------------------------------------------------- rows to int8

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 8), (3, 16), (7, 264), (1, 2816), (33, 704), (130, 1032),
                                    (9, 4096), (5, 8200), (2, 20000), (1000, 512)])
def test_quantize_rows(rows, K, dt):
    rng = np.random.default_rng(rows * 1000 + K)
    x, xv = rounded(rng.standard_normal((rows, K)) * np.exp(rng.uniform(-20, 20, (rows, 1))), dt)
    q, s = moe.quantize_rows(x.cuda())
    rq, rs = O.quantize_rows(xv)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_rows_at_halves(dt):
    """Rows whose quotients are halves, or one ulp to either side of one."""
    top = np.float32(127.0 if dt == "bf16" else 127.0 * 3)
    halves = (np.arange(0, 127) + 0.5) * (1.0 if dt == "bf16" else 3.0)
    rows = []
    for sign in (1, -1):
        for step in (0, 1, -1):
            v = np.asarray(halves * sign, dtype=np.float32)
            if step and dt == "f32":
                v = np.nextafter(v, np.float32(np.inf * step)).astype(np.float32)
            rows.append(np.concatenate([v, [top]]))
    x, xv = rounded(np.array(rows), dt)
    q, s = moe.quantize_rows(x.cuda())
    rq, rs = O.quantize_rows(xv)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_rows_extremes(dt):
    """Zeros, subnormals, the type's largest values, infinities and NaN, one to a row."""
    big = float(torch.finfo(TORCH[dt]).max)
    rng = np.random.default_rng(5)
    base = rng.uniform(-1, 1, 24)
    with np.errstate(over="ignore"):
        x = np.array([np.zeros(24), base * 1e-39, base * 1e-44, base * big, np.full(24, -big), base * 2e-31,
                      base * 2e37, base, base, base, -np.zeros(24)], dtype=np.float32)
    x[7, 3], x[8, 0], x[9, 23] = np.inf, np.nan, -np.inf
    t, xv = rounded(x, dt)
    q, s = moe.quantize_rows(t.cuda())
    rq, rs = O.quantize_rows(xv)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)


# ------------------------------------------------------------------------------- products

PRODUCTS = [  # rows, K, N, E (0: dense), used experts
    (1, 16, 32, 0, None), (1, 2816, 1408, 0, None), (2, 144, 96, 0, None), (17, 128, 160, 0, None),
    (64, 704, 256, 0, None), (65, 272, 288, 0, None), (129, 400, 544, 0, None), (300, 1040, 512, 0, None),
    (777, 256, 1312, 0, None), (1, 64, 64, 3, None), (32, 256, 192, 16, None), (40, 2816, 96, 5, 2),
    (257, 192, 320, 4, None), (700, 320, 256, 7, 3), (2000, 128, 416, 256, None), (900, 528, 224, 2, 1),
    (3000, 1152, 1056, 0, None), (2100, 832, 1504, 9, 6),   # CTA pairs, K of more than six blocks
]


def _product_case(rows, K, N, E, used, dt, bias, seed):
    rng = np.random.default_rng(seed)
    x, xv = rounded(rng.standard_normal((rows, K)), dt)
    n = [rows] if not E else split(rows, E, rng, used=used)
    w, ws = weights(rng, max(E, 1), N, K)
    b = bv = None
    if bias:
        b, bv = rounded(rng.standard_normal((max(E, 1), N)), dt)
    return x, xv, np.concatenate([[0], np.cumsum(n)]).astype(np.int32), w, ws, b, bv


def _product_ref(xv, off, w, ws, bv, dt, rows, N):
    q, s = O.quantize_rows(xv)
    y, bound = np.zeros((rows, N)), np.zeros((rows, N))
    for e in range(len(off) - 1):
        a, z = off[e], off[e + 1]
        if a < z:
            y[a:z] = O.matmul_q8(q[a:z], s[a:z], w[e], ws[e], None if bv is None else bv[e])
            bound[a:z] = product_bound(q[a:z], s[a:z], w[e], ws[e], y[a:z], dt)
    return y, bound


@pytest.mark.parametrize("dt,bias", [("bf16", False), ("f32", True), ("bf16", True)])
@pytest.mark.parametrize("rows,K,N,E,used", PRODUCTS)
def test_matmul_q8(rows, K, N, E, used, dt, bias):
    x, xv, off, w, ws, b, bv = _product_case(rows, K, N, E, used, dt, bias, rows + K + N)
    q, s = moe.quantize_rows(x.cuda())
    b = None if b is None else b.cuda()
    if E:
        out = moe.matmul_q8(q, s, dev(w), dev(ws), offsets=dev(off), bias=b, out_dtype=TORCH[dt])
    else:
        out = moe.matmul_q8(q, s, dev(w[0]), dev(ws[0]), bias=None if b is None else b[0], out_dtype=TORCH[dt])
    y, bound = _product_ref(xv, off, w, ws, bv, dt, rows, N)
    check(from_dev(out), y, bound, f"product {rows}x{K}x{N} E={E}")


@pytest.mark.parametrize("rows,K,N,E,used,dt,bias", [
    (20000, 16, 3104, 0, None, "bf16", True), (9001, 704, 6240, 0, None, "bf16", False),
    (30000, 272, 1824, 3, 2, "f32", True), (12000, 768, 5152, 5, None, "bf16", True),
    (24000, 80, 4768, 4, 3, "f32", False), (24001, 400, 4800, 60, 50, "bf16", True),
])
def test_matmul_q8_weights_kept_for_several_token_tiles(rows, K, N, E, used, dt, bias):
    """Sizes at which a CTA pair keeps a weight tile for 2 to 4 token tiles (K of one to six
    128-wide blocks, ragged tiles and groups, experts without rows)."""
    x, xv, off, w, ws, b, bv = _product_case(rows, K, N, E, used, dt, bias, rows + K)
    q, s = moe.quantize_rows(x.cuda())
    b = None if b is None else b.cuda()
    if E:
        out = moe.matmul_q8(q, s, dev(w), dev(ws), offsets=dev(off), bias=b, out_dtype=TORCH[dt])
    else:
        out = moe.matmul_q8(q, s, dev(w[0]), dev(ws[0]), bias=None if b is None else b[0], out_dtype=TORCH[dt])
    y, bound = _product_ref(xv, off, w, ws, bv, dt, rows, N)
    check(from_dev(out), y, bound, f"product {rows}x{K}x{N} E={E}")


def test_matmul_q8_largest_sums():
    """Every product at its largest, K at its limit: 127^2 K and 127 * 128 K in int32."""
    K = 65536
    a = torch.full((3, K), 127, dtype=torch.int8, device="cuda")
    w = torch.full((64, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one_a, one_w = torch.ones(3, device="cuda"), torch.ones(64, device="cuda")
    out = moe.matmul_q8(a, one_a, w, one_w, out_dtype=torch.float32).cpu()
    assert torch.all(out[:, 0::2] == -127.0 * 128 * K) and torch.all(out[:, 1::2] == 127.0 * 127 * K)


@pytest.mark.parametrize("rows,E", [(40, 4), (600, 4)])
def test_rows_behind_the_last_expert_stay_as_they_were(rows, E):
    x, xv, off, w, ws, _, _ = _product_case(rows, 256, 128, E, None, "bf16", False, 3)
    off = np.minimum(off, rows - 7).astype(np.int32)
    q, s = moe.quantize_rows(x.cuda())
    out = torch.full((rows, 128), 42.0, dtype=torch.bfloat16, device="cuda")
    moe.matmul_q8(q, s, dev(w), dev(ws), offsets=dev(off), out=out)
    y, bound = _product_ref(xv, off, w, ws, None, "bf16", rows, 128)
    check(from_dev(out)[:rows - 7], y[:rows - 7], bound[:rows - 7], "rows of the experts")
    assert torch.all(out[rows - 7:] == 42.0)


def test_bad_offsets_are_clamped_and_reported():
    x, _, off, w, ws, _, _ = _product_case(64, 256, 128, 4, None, "bf16", False, 4)
    q, s = moe.quantize_rows(x.cuda())
    for bad in ([0, 10, 5, 20, 64], [0, 10, 20, 30, 1000], [-3, 10, 20, 30, 64]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.matmul_q8(q, s, dev(w), dev(ws), offsets=dev(np.array(bad, dtype=np.int32)), err_word=err)
        assert moe.get_error(err) == (_abi.MOE_ERR_DEVICE, 1), bad
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.matmul_q8(q, s, dev(w), dev(ws), offsets=dev(off), err_word=err)
    assert moe.get_error(err) == (_abi.MOE_OK, 0)


def test_nan_rows_stay_in_their_rows():
    """A row with an infinity or a NaN comes out NaN, its neighbours as without it."""
    x, xv, off, w, ws, _, _ = _product_case(70, 256, 128, 3, None, "f32", False, 6)
    xd = x.cuda()
    q, s = moe.quantize_rows(xd)
    ref = moe.matmul_q8(q, s, dev(w), dev(ws), offsets=dev(off), out_dtype=torch.float32)
    xd[5, 7], xd[44, 0] = float("nan"), float("inf")
    q, s = moe.quantize_rows(xd)
    out = moe.matmul_q8(q, s, dev(w), dev(ws), offsets=dev(off), out_dtype=torch.float32)
    keep = [r for r in range(70) if r not in (5, 44)]
    assert torch.isnan(out[[5, 44]]).all() and torch.equal(out[keep], ref[keep])


# ------------------------------------------------------------------------------------ FFN

FFNS = [  # rows, H, I, E, used, layout, act, biases
    (1, 32, 32, 1, None, "interleaved", STD, False),
    (8, 256, 128, 4, None, "interleaved", STD, False),
    (32, 2816, 704, 6, 3, "interleaved", STD, False),
    (33, 288, 96, 8, None, "chunked", OSS, True),
    (64, 64, 32, 2, 1, "chunked", STD, True),
    (200, 352, 160, 3, None, "interleaved", OSS, True),
    (500, 256, 224, 2, 1, "chunked", STD, False),
    (1100, 512, 256, 3, None, "interleaved", STD, True),
    (900, 384, 704, 200, None, "chunked", OSS, False),
    # many rows of short K: fc1's, or fc2's, weight tiles kept for several token tiles
    (30000, 64, 1024, 3, 2, "chunked", OSS, True), (30000, 1824, 64, 2, None, "interleaved", STD, False),
]


def _ffn_case(rows, H, I, E, used, biases, seed):
    rng = np.random.default_rng(seed)
    x, xv = rounded(rng.standard_normal((rows, H)), "bf16")
    off = np.concatenate([[0], np.cumsum(split(rows, E, rng, used=used))]).astype(np.int32)
    q1, s1 = weights(rng, E, 2 * I, H)
    q2, s2 = weights(rng, E, H, I)
    b1 = b2 = (None, None)
    if biases:
        b1, b2 = rounded(rng.standard_normal((E, 2 * I)) * 0.5, "bf16"), rounded(rng.standard_normal((E, H)) * 0.5, "bf16")
    return x.cuda(), xv, off, q1, s1, q2, s2, b1, b2


def _ffn_ref(xv, off, q1, s1, q2, s2, b1v, b2v, layout, act):
    y, bound = np.zeros(xv.shape), np.zeros(xv.shape)
    for e in range(len(off) - 1):
        a, z = off[e], off[e + 1]
        if a < z:
            y[a:z], bound[a:z] = ffn_with_bound(xv[a:z], q1[e], s1[e], q2[e], s2[e], layout, act,
                                                None if b1v is None else b1v[e], None if b2v is None else b2v[e])
    return y, bound


def _dev_bias(b):
    return None if b[0] is None else b[0].cuda()


@pytest.mark.parametrize("rows,H,I,E,used,layout,act,biases", FFNS)
def test_expert_ffn_w8a8(rows, H, I, E, used, layout, act, biases):
    x, xv, off, q1, s1, q2, s2, b1, b2 = _ffn_case(rows, H, I, E, used, biases, rows + H)
    y = moe.expert_ffn_w8a8(x, dev(off), dev(q1), dev(s1), dev(q2), dev(s2), swiglu=act, fc1_layout=layout,
                            fc1_bias=_dev_bias(b1), fc2_bias=_dev_bias(b2))
    ref, bound = _ffn_ref(xv, off, q1, s1, q2, s2, b1[1], b2[1], layout, act)
    check(from_dev(y), ref, bound, f"ffn {rows}x{H}x{I} E={E}")


@pytest.mark.parametrize("rows", [24, 640])
def test_expert_ffn_w8a8_workspace_reuse_tail_and_errors(rows):
    """One workspace with any contents serves calls in a row; rows behind the last expert
    keep their values; bad offsets are reported in the workspace's first word."""
    H, I, E = 256, 128, 4
    x, xv, off, q1, s1, q2, s2, _, _ = _ffn_case(rows, H, I, E, None, False, 9)
    off = np.minimum(off, rows - 5).astype(np.int32)
    nb = moe.expert_ffn_w8a8_workspace_size(rows, H, E, I)
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda")
    w = [dev(a) for a in (q1, s1, q2, s2)]
    ys = []
    for _ in range(3):
        y = torch.full((rows, H), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.expert_ffn_w8a8(x, dev(off), *w, y_perm=y, workspace=ws)
        assert moe.get_error(moe.workspace_error_word(ws)) == (_abi.MOE_OK, 0)
        assert torch.all(y[rows - 5:] == 7.0)
        ys.append(y)
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])
    ref, bound = _ffn_ref(xv, off, q1, s1, q2, s2, None, None, "interleaved", STD)
    check(from_dev(ys[0])[:rows - 5], ref[:rows - 5], bound[:rows - 5], "ffn")
    bad = off.copy()
    bad[2] = rows + 100
    moe.expert_ffn_w8a8(x, dev(bad), *w, workspace=ws)
    assert moe.get_error(moe.workspace_error_word(ws)) == (_abi.MOE_ERR_DEVICE, 1)


@pytest.mark.parametrize("rows", [16, 600])
def test_expert_ffn_w8a8_nan_row_and_zero_row(rows):
    H, I, E = 128, 64, 2
    x, xv, off, q1, s1, q2, s2, _, _ = _ffn_case(rows, H, I, E, None, False, 10)
    w = [dev(a) for a in (q1, s1, q2, s2)]
    ref = moe.expert_ffn_w8a8(x, dev(off), *w)
    x2 = x.clone()
    x2[3, 5] = float("nan")
    x2[9] = 0
    y = moe.expert_ffn_w8a8(x2, dev(off), *w)
    keep = [r for r in range(rows) if r not in (3, 9)]
    assert torch.isnan(y[3].float()).all() and torch.all(y[9] == 0) and torch.equal(y[keep], ref[keep])


# ---------------------------------------------------------------------------------- layer

def W(name, **kw):
    base = dict(T=64, H=128, E=8, k=2, I=64, dtype="bf16", seed=1)
    base.update(kw)
    return Workload(name, **base)


LAYERS = [W("one_token", T=1, H=512, E=64, k=8, I=192), W("small", T=5, H=256, E=16, k=4, I=128),
          W("tc_router", T=100, H=256, E=64, k=4, I=192, router_bias_std=0.5),
          W("chunked_norm0", T=20, H=256, E=32, k=6, I=128, normalize=0, fc1_layout="chunked"),
          W("prefill", T=700, H=256, E=8, k=2, I=96), W("k40", T=30, H=128, E=64, k=40, I=64)]


@pytest.mark.parametrize("wl", LAYERS, ids=[w.name for w in LAYERS])
def test_forward_w8a8(wl):
    """The layer equals its steps called one by one, bit for bit, and the weight-only int8
    layer up to the rounding of the activations to 8 bits (a loose check of the wiring)."""
    inp = make_inputs(wl, weights=False)
    d = device_inputs(inp)
    host = make_q8_experts(wl, None)
    q1, s1, q2, s2 = [dev(a) for a in host]
    kw = dict(normalize=bool(wl.normalize), router_bias=d["router_bias"])
    out = moe.forward_w8a8(d["hidden"], d["router_w"], q1, s1, q2, s2, wl.k, fc1_layout=wl.fc1_layout, **kw)
    r = moe.route(d["hidden"], d["router_w"], wl.k, **kw)
    L = O.router_logits(inp.values("hidden"), inp.values("router_w"), inp["router_bias"])
    idx, _ = match_routing(L, from_dev(r["idx"]).astype(np.int64), wl.k)
    ref = O.moe_forward(inp.values("hidden"), inp.values("router_w"), inp["router_bias"],
                        lambda e: O.dequantize_rows(host[0][e], host[1][e]),
                        lambda e: O.dequantize_rows(host[2][e], host[3][e]), wl.k, wl.normalize,
                        wl.fc1_layout, idx=idx)["out"]
    got = from_dev(out)
    assert np.linalg.norm(got - ref) < 0.05 * np.linalg.norm(ref)
    p = moe.permute(r["idx"], wl.E, hidden=d["hidden"])
    y = moe.expert_ffn_w8a8(p["x_perm"], p["offsets"], q1, s1, q2, s2, fc1_layout=wl.fc1_layout)
    c = moe.combine(y, p["perm_dst"], r["w"], wl.T, wl.k)
    if wl.T > 16 and wl.name != "chunked_norm0" and wl.k <= 32:
        assert torch.equal(out, c)
    else:
        # the layer and moe_route take different routers here (float32 sums in another
        # order): weights within 1e-5, an output within that of the experts' magnitudes
        assert_close(got, from_dev(c), 1e-5 * wl.k * float(y.float().abs().max()), 2.0 ** -7, wl.name)


def test_forward_w8a8_with_pre_norm_and_workspace():
    wl = W("norm", T=40, H=256, E=16, k=4, I=128)
    inp = make_inputs(wl, weights=False)
    d = device_inputs(inp)
    q1, s1, q2, s2 = [dev(a) for a in make_q8_experts(wl, None)]
    rng = np.random.default_rng(0)
    nw, _ = rounded(rng.uniform(0.5, 1.5, wl.H), "bf16")
    ws = torch.full((moe.w8a8_workspace_size(wl.T, wl.H, wl.E, wl.k, wl.I),), 0x5A, dtype=torch.uint8, device="cuda")
    a = moe.forward_w8a8(d["hidden"], d["router_w"], q1, s1, q2, s2, wl.k, norm_weight=nw.cuda(), workspace=ws)
    assert moe.get_error(moe.workspace_error_word(ws)) == (_abi.MOE_OK, 0)
    xn = moe.rmsnorm(d["hidden"], nw.cuda())
    b = moe.forward_w8a8(xn, d["router_w"], q1, s1, q2, s2, wl.k, workspace=ws)
    assert torch.equal(a, b)


# ------------------------------------------------------------------------ how it is called

def test_on_another_stream_and_captured():
    """A run of the calls on a side stream, captured and replayed on new inputs."""
    H, I, E, rows = 256, 128, 4, 48
    x, xv, off, q1, s1, q2, s2, _, _ = _ffn_case(rows, H, I, E, None, False, 12)
    w = [dev(a) for a in (q1, s1, q2, s2)]
    o = dev(off)
    eager = moe.expert_ffn_w8a8(x, o, *w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = moe.expert_ffn_w8a8(x, o, *w, stream=side)
    side.synchronize()
    assert torch.equal(y, eager)
    xin, yout = torch.zeros_like(x), torch.zeros_like(x)
    ws = torch.empty(moe.expert_ffn_w8a8_workspace_size(rows, H, E, I), dtype=torch.uint8, device="cuda")
    graphs = []
    for _ in range(2):   # two graphs that share the workspace, replayed one after the other
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q, s = moe.quantize_rows(xin)
            prod = moe.matmul_q8(q, s, w[0], w[1], offsets=o)
            moe.expert_ffn_w8a8(xin, o, *w, y_perm=yout, workspace=ws)
        graphs.append((g, prod))
    for i in range(4):
        xin.copy_(x if i % 2 == 0 else -x)
        g, prod = graphs[i % 2]
        g.replay()
        torch.cuda.synchronize()
        want = moe.expert_ffn_w8a8(xin, o, *w)
        q, s = moe.quantize_rows(xin)
        assert torch.equal(yout, want) and torch.equal(prod, moe.matmul_q8(q, s, w[0], w[1], offsets=o))


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its own workspace."""
    rows, H, I, E = 400, 512, 256, 4
    x, xv, off, q1, s1, q2, s2, _, _ = _ffn_case(rows, H, I, E, None, False, 13)
    w = [dev(a) for a in (q1, s1, q2, s2)]
    o = dev(off)
    want = moe.expert_ffn_w8a8(x, o, *w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            ys[i].append(moe.expert_ffn_w8a8(x, o, *w, stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        for y in ys[i]:
            assert torch.equal(y, want)


def test_binding_refuses_mismatches():
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    q, s = moe.quantize_rows(x)
    w, sw = torch.zeros(32, 64, dtype=torch.int8, device="cuda"), torch.zeros(32, device="cuda")
    with pytest.raises(ValueError):
        moe.matmul_q8(q, s, w[None], sw)                       # grouped weights without offsets
    with pytest.raises(ValueError):
        moe.matmul_q8(q.t(), s, w, sw)                         # not contiguous
    with pytest.raises(TypeError):
        moe.matmul_q8(q, s, w.float(), sw)
    with pytest.raises(TypeError):
        moe.matmul_q8(q, s, w, sw, bias=torch.zeros(32, device="cuda"))   # float32 bias, bf16 out
    with pytest.raises(ValueError):
        moe.matmul_q8(q, s, w, sw, out=torch.zeros(8, 33, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        moe.quantize_rows(x.half())
    with pytest.raises(moe.MoEError):
        moe.quantize_rows(torch.zeros(2, 12, device="cuda"))   # K not a multiple of 8
    with pytest.raises(moe.MoEError):
        moe.matmul_q8(q[:, :24].contiguous(), s, w[:, :24].contiguous(), sw)


# The kernel of few rows, which runs the whole FFN in one launch: at fewer than 8 rows an
# expert, and up to 48 where fc1 alone has more units of 256 weight rows than the chip has SMs.
FEW = [  # rows, H, I, E, used, layout, act, biases
    (12, 128, 64, 2, None, "interleaved", STD, False),
    (20, 256, 128, 4, None, "chunked", OSS, True),
    (900, 256, 96, 200, 3, "interleaved", STD, True),      # several chunks of one expert's tokens
    (1500, 544, 416, 40, 2, "chunked", STD, False),        # more than 8 rows an expert, all in two
    (1000, 160, 320, 50, 45, "interleaved", OSS, True),
    (5, 32, 32, 256, None, "interleaved", STD, False),
]


@pytest.mark.parametrize("rows,H,I,E,used,layout,act,biases", FEW)
def test_expert_ffn_w8a8_in_one_launch(rows, H, I, E, used, layout, act, biases):
    x, xv, off, q1, s1, q2, s2, b1, b2 = _ffn_case(rows, H, I, E, used, biases, rows + I)
    y = moe.expert_ffn_w8a8(x, dev(off), dev(q1), dev(s1), dev(q2), dev(s2), swiglu=act, fc1_layout=layout,
                            fc1_bias=_dev_bias(b1), fc2_bias=_dev_bias(b2))
    ref, bound = _ffn_ref(xv, off, q1, s1, q2, s2, b1[1], b2[1], layout, act)
    check(from_dev(y), ref, bound, f"ffn {rows}x{H}x{I} E={E}")


def test_few_rows_nan_row_and_zero_row():
    rows, H, I, E = 14, 128, 64, 4
    x, xv, off, q1, s1, q2, s2, _, _ = _ffn_case(rows, H, I, E, None, False, 20)
    w = [dev(a) for a in (q1, s1, q2, s2)]
    ref = moe.expert_ffn_w8a8(x, dev(off), *w)
    x2 = x.clone()
    x2[3, 5] = float("inf")
    x2[9] = 0
    y = moe.expert_ffn_w8a8(x2, dev(off), *w)
    keep = [r for r in range(rows) if r not in (3, 9)]
    assert torch.isnan(y[3].float()).all() and torch.all(y[9] == 0) and torch.equal(y[keep], ref[keep])


@pytest.mark.parametrize("rows", [20, 400])
def test_no_rows_in_any_expert(rows):
    """Offsets that give no expert a row: nothing is written, no error."""
    x, xv, off, q1, s1, q2, s2, _, _ = _ffn_case(rows, 128, 64, 4, None, False, 21)
    w = [dev(a) for a in (q1, s1, q2, s2)]
    nb = moe.expert_ffn_w8a8_workspace_size(rows, 128, 4, 64)
    ws = torch.full((nb,), 0xA5, dtype=torch.uint8, device="cuda")
    y = torch.full((rows, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    moe.expert_ffn_w8a8(x, torch.zeros(5, dtype=torch.int32, device="cuda"), *w, y_perm=y, workspace=ws)
    assert moe.get_error(moe.workspace_error_word(ws)) == (_abi.MOE_OK, 0) and torch.all(y == 3.0)


def test_few_rows_two_streams_and_graphs():
    """The one-launch FFN on two streams at once, and two graphs that share a workspace."""
    rows, H, I, E = 20, 512, 256, 4
    x, xv, off, q1, s1, q2, s2, _, _ = _ffn_case(rows, H, I, E, None, False, 22)
    w = [dev(a) for a in (q1, s1, q2, s2)]
    o = dev(off)
    want = {1: moe.expert_ffn_w8a8(x, o, *w), -1: moe.expert_ffn_w8a8(-x, o, *w)}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [moe.expert_ffn_w8a8(x, o, *w, stream=streams[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[1]) for y in ys)
    xin, yout = torch.zeros_like(x), torch.zeros_like(x)
    ws = torch.empty(moe.expert_ffn_w8a8_workspace_size(rows, H, E, I), dtype=torch.uint8, device="cuda")
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            for _ in range(3):   # calls in a row: each clears what the one before left
                moe.expert_ffn_w8a8(xin, o, *w, y_perm=yout, workspace=ws)
    for i in range(6):
        sign = 1 if i % 2 == 0 else -1
        xin.copy_(sign * x)
        graphs[i % 2].replay()
        assert torch.equal(yout, want[sign])


@pytest.mark.parametrize("rows,H,I,E,empty", [(25, 256, 96, 3, 9), (100, 352, 160, 4, 30), (700, 64, 224, 2, 150)])
def test_experts_without_rows_change_nothing(rows, H, I, E, empty):
    """The same rows with and without experts that get none: other kernels (the launches of
    many rows per expert, the one of few), the same bits."""
    x, _, off, q1, s1, q2, s2, b1, b2 = _ffn_case(rows, H, I, E, None, True, 23)
    w = [dev(a) for a in (q1, s1, q2, s2)]
    want = moe.expert_ffn_w8a8(x, dev(off), *w, swiglu=OSS, fc1_bias=b1[0].cuda(), fc2_bias=b2[0].cuda())

    def spread(t):   # every expert behind `empty` / E others of the same size
        out = torch.ones((E, empty // E + 1) + t.shape[1:], dtype=t.dtype, device="cuda")
        out[:, -1] = t
        return out.flatten(0, 1).contiguous()
    step = empty // E + 1
    many = np.concatenate([[0], np.repeat(off[1:], step)])
    for e in range(E):
        many[1 + e * step:1 + (e + 1) * step - 1] = off[e]
    y = moe.expert_ffn_w8a8(x, dev(many.astype(np.int32)), *[spread(t) for t in w], swiglu=OSS,
                            fc1_bias=spread(b1[0].cuda()), fc2_bias=spread(b2[0].cuda()))
    assert torch.equal(y, want)
