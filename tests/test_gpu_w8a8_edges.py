"""int8 rows, products and expert FFN on the GPU at the edges of what their contracts allow:
rows that are not finite under every activation, empty calls, very many rows, long
intermediate sizes in the one-launch FFN.  Bounds: w8a8_util."""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_15_b200 as moe
from mixture_experts_ffn_15_b200 import _abi
from parity_util import from_dev
from test_gpu_w8a8 import OSS, STD, _dev_bias, _ffn_case, _ffn_ref, dev
from w8a8_util import check

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


# rows, E: the one launch of few rows per expert, and the separate launches of many
@pytest.mark.parametrize("rows,E", [(14, 4), (16, 2), (600, 2)])
@pytest.mark.parametrize("act", [STD, OSS, (1.0, 0.0, 0.5)], ids=["standard", "gpt_oss", "clipped"])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("layout", ["interleaved", "chunked"])
def test_a_row_that_is_not_finite_comes_out_nan(rows, E, act, value, layout):
    """Its scale is NaN, so every gate and up value is: the clip carries that on."""
    H, I = 128, 64
    x, _, off, q1, s1, q2, s2, b1, b2 = _ffn_case(rows, H, I, E, None, True, 30)
    args = [dev(off)] + [dev(a) for a in (q1, s1, q2, s2)]
    kw = dict(swiglu=act, fc1_layout=layout, fc1_bias=b1[0].cuda(), fc2_bias=b2[0].cuda())
    ref = moe.expert_ffn_w8a8(x, *args, **kw)
    x2 = x.clone()
    x2[3, 5] = value
    y = moe.expert_ffn_w8a8(x2, *args, **kw)
    keep = [r for r in range(rows) if r != 3]
    assert torch.isnan(y[3].float()).all() and torch.equal(y[keep], ref[keep])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [14, 600])
def test_a_nan_row_of_the_unquantised_ffn_comes_out_nan(rows, dt):
    """The same clip in the bf16 and float32 experts."""
    H, I, E = 128, 64, 2
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn((rows, H), generator=g, device="cuda").to(dt)
    w1 = (torch.randn((E, 2 * I, H), generator=g, device="cuda") / H ** 0.5).to(dt)
    w2 = (torch.randn((E, H, I), generator=g, device="cuda") / I ** 0.5).to(dt)
    off = torch.tensor([0, rows // 2, rows], dtype=torch.int32, device="cuda")
    ref = moe.expert_ffn(x, off, w1, w2, swiglu=OSS)
    x[3, 5] = NAN
    y = moe.expert_ffn(x, off, w1, w2, swiglu=OSS)
    keep = [r for r in range(rows) if r != 3]
    assert torch.isnan(y[3].float()).all() and torch.equal(y[keep], ref[keep])


def test_a_nan_row_of_the_weight_only_int8_ffn_comes_out_nan():
    rows, H, I, E = 14, 128, 128, 2
    x, _, off, q1, s1, q2, s2, _, _ = _ffn_case(rows, H, I, E, None, False, 32)
    args = [dev(off)] + [dev(a) for a in (q1, s1, q2, s2)]
    ref = moe.expert_ffn_q8(x, *args, swiglu=OSS)
    x[3, 5] = NAN
    y = moe.expert_ffn_q8(x, *args, swiglu=OSS)
    keep = [r for r in range(rows) if r != 3]
    assert torch.isnan(y[3].float()).all() and torch.equal(y[keep], ref[keep])


def test_quantize_rows_of_more_than_2_31_threads():
    """2^26 + 3 rows of 8 values: 32 threads a row, so that the thread numbers pass 31 bits."""
    rows, K, step = (1 << 26) + 3, 8, 1 << 23
    g = torch.Generator(device="cuda").manual_seed(33)
    x = torch.empty((rows, K), dtype=torch.bfloat16, device="cuda")
    for a in range(0, rows, step):
        x[a:a + step].normal_(generator=g)
    q, s = moe.quantize_rows(x)
    for a in range(0, rows, step):
        v = x[a:a + step].double()
        top = v.abs().amax(1, keepdim=True)
        # by a tensor: torch multiplies by the reciprocal of a Python number
        assert torch.equal(s[a:a + step], top[:, 0].float() / torch.full_like(s[a:a + step], 127))
        # 127 v is exact in float64, the quotient is a half exactly or far from one
        assert torch.equal(q[a:a + step], (127 * v / top.clamp_min(1e-300)).round().to(torch.int8))


@pytest.mark.parametrize("stream", [False, True])
def test_the_error_word_of_an_empty_call_is_zero(stream):
    """A workspace may hold anything; so may the last call's error."""
    _, _, _, q1, s1, q2, s2, _, _ = _ffn_case(8, 64, 32, 4, None, False, 34)
    w = [dev(a) for a in (q1, s1, q2, s2)]
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    router = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    for n, call in ((moe.expert_ffn_w8a8_workspace_size(0, 64, 4, 32), lambda **kw: moe.expert_ffn_w8a8(x, off, *w, **kw)),
                    (moe.w8a8_workspace_size(0, 64, 4, 2, 32), lambda **kw: moe.forward_w8a8(x, router, *w, 2, **kw))):
        ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        st = torch.cuda.Stream() if stream else None
        y = call(workspace=ws, stream=st)
        torch.cuda.synchronize()
        assert y.shape == (0, 64) and moe.get_error(moe.workspace_error_word(ws)) == (_abi.MOE_OK, 0)
        assert torch.all(ws[4:] == 0xA5)


# The one launch's rounding holds 1024 values of a row in registers and reads the rest again.
LONG = [  # rows, H, I, E, used, layout, act, biases
    (20, 64, 1056, 4, None, "interleaved", STD, False),
    (9, 96, 2080, 2, None, "chunked", OSS, True),
    (500, 64, 1216, 80, 5, "chunked", STD, True),          # several chunks an expert, odd ends
    (3, 32, 4128, 1, None, "interleaved", OSS, False),
    (7, 128, 1024, 1, None, "interleaved", STD, False),
    (33, 160, 992, 5, 2, "chunked", OSS, False),
]


@pytest.mark.parametrize("rows,H,I,E,used,layout,act,biases", LONG)
def test_one_launch_with_long_activation_rows(rows, H, I, E, used, layout, act, biases):
    x, xv, off, q1, s1, q2, s2, b1, b2 = _ffn_case(rows, H, I, E, used, biases, rows + I)
    y = moe.expert_ffn_w8a8(x, dev(off), dev(q1), dev(s1), dev(q2), dev(s2), swiglu=act, fc1_layout=layout,
                            fc1_bias=_dev_bias(b1), fc2_bias=_dev_bias(b2))
    ref, bound = _ffn_ref(xv, off, q1, s1, q2, s2, b1[1], b2[1], layout, act)
    check(from_dev(y), ref, bound, f"ffn {rows}x{H}x{I} E={E}")


@pytest.mark.parametrize("at", [5, 1023, 1024, 1500, 2079])
def test_one_launch_with_the_largest_activation_anywhere_in_its_row(at):
    """One channel's scale raised 64-fold: its activations are the rows' largest."""
    rows, H, I, E = 9, 96, 2080, 2
    x, xv, off, q1, s1, q2, s2, _, _ = _ffn_case(rows, H, I, E, None, False, 35)
    s1[:, 2 * at + 1] *= 64          # interleaved: the channel's up row
    y = moe.expert_ffn_w8a8(x, dev(off), dev(q1), dev(s1), dev(q2), dev(s2))
    ref, bound = _ffn_ref(xv, off, q1, s1, q2, s2, None, None, "interleaved", STD)
    check(from_dev(y), ref, bound, f"largest at {at}")


@pytest.mark.parametrize("T,E,k,layout", [(1, 16, 4, "interleaved"), (6, 64, 8, "chunked"), (90, 8, 2, "interleaved"),
                                          (700, 8, 2, "chunked"), (900, 60, 4, "interleaved")])
@pytest.mark.parametrize("norm", [False, True])
def test_the_layer_with_biases_and_a_clipped_activation_equals_its_steps(T, E, k, layout, norm):
    """forward_w8a8 with every option against rmsnorm, route, permute, expert_ffn_w8a8 and
    combine.  The layer and moe_route may take different routers (float32 sums in another order):
    weights within 1e-5, an output within that of the experts' magnitudes."""
    H, I = 256, 96
    rng = np.random.default_rng(T)
    x, _, _, q1, s1, q2, s2, b1, b2 = _ffn_case(T, H, I, E, None, True, 36)
    w = [dev(a) for a in (q1, s1, q2, s2)]
    router = torch.from_numpy(rng.standard_normal((E, H)) / 16).bfloat16().cuda()
    rb = torch.from_numpy((rng.standard_normal(E) * 0.3).astype(np.float32)).cuda()
    nw = torch.from_numpy(rng.uniform(0.5, 1.5, H)).bfloat16().cuda() if norm else None
    ffn = dict(swiglu=OSS, fc1_layout=layout, fc1_bias=b1[0].cuda(), fc2_bias=b2[0].cuda())
    out = moe.forward_w8a8(x, router, *w, k, router_bias=rb, norm_weight=nw, **ffn)
    xn = moe.rmsnorm(x, nw) if norm else x
    r = moe.route(xn, router, k, router_bias=rb)
    p = moe.permute(r["idx"], E, hidden=xn)
    y = moe.expert_ffn_w8a8(p["x_perm"], p["offsets"], *w, **ffn)
    want = moe.combine(y, p["perm_dst"], r["w"], T, k)
    sure = r["near_tie"] == 0
    d = (out.double() - want.double()).abs()
    assert torch.all(d[sure] <= 1e-5 * k * float(y.float().abs().max()) + 2.0 ** -7 * want[sure].double().abs())
    assert int(sure.sum()) > 0
