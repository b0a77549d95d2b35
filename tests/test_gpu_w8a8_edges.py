"""int8 rows, products and expert FFN on the GPU at the edges of what their contracts allow:
rows that are not finite under every activation, empty calls, very many rows, long
intermediate sizes in the one-launch FFN.  Bounds: w8a8_util."""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_15_b200 as moe
from mixture_experts_ffn_15_b200 import _abi
from test_gpu_w8a8 import OSS, STD, _ffn_case, dev

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
