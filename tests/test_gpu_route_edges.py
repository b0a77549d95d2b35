"""Routing of tokens with fewer than k logits above -infinity (experts masked by the router
bias, rows that are not finite) by each router: ids stay valid, other tokens are untouched."""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_15_b200 as moe
from mixture_experts_ffn_15_b200 import _abi
from oracle import moe_oracle as O
from parity_util import from_dev

pytestmark = pytest.mark.gpu

# T, E, k: one CTA, split over K in clusters, a CTA a tile (E = 256; many tiles), SIMT
SIZES = [(5, 64, 8), (20, 64, 8), (300, 128, 8), (300, 128, 20), (40, 256, 8), (130, 256, 30), (20000, 64, 2),
         (700, 60, 4), (30, 64, 40), (600, 7, 7)]
H, I = 128, 64


def inputs(T, E, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    w = (torch.randn((E, H), generator=g, device="cuda") / 8).bfloat16()
    q1 = torch.randint(-127, 128, (E, 2 * I, H), dtype=torch.int8, device="cuda", generator=g)
    q2 = torch.randint(-127, 128, (E, H, I), dtype=torch.int8, device="cuda", generator=g)
    s1 = torch.full((E, 2 * I), 1e-3, device="cuda")
    s2 = torch.full((E, H), 1e-3, device="cuda")
    return x, w, q1, s1, q2, s2


def valid(idx, E):
    i = idx.cpu().numpy()
    assert i.min() >= 0 and i.max() < E
    assert all(len(set(row)) == len(row) for row in i[:400])


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_fewer_than_k_experts_left_by_the_bias(T, E, k, normalize):
    """The masked experts fill the list in index order with weight 0."""
    x, w, q1, s1, q2, s2 = inputs(T, E, 1)
    bias = torch.full((E,), float("-inf"), device="cuda")
    left = [E - 1, 2, E // 2][:max(k - 1, 1)]
    bias[left] = 0.25
    r = moe.route(x, w, k, normalize=normalize, router_bias=bias)
    valid(r["idx"], E)
    L = O.router_logits(from_dev(x[:64]), from_dev(w), bias.cpu().numpy())
    i, n = r["idx"][:64].cpu().numpy(), min(k, len(left))
    assert all(set(row[:n]) <= set(left) for row in i)
    if k > len(left):
        rest = [e for e in range(E) if e not in left][:k - len(left)]
        assert np.all(i[:, len(left):] == rest) and not r["w"][:, len(left):].any()
    for t in range(min(T, 64)):
        p = np.exp(L[t, i[t]] - L[t].max())
        p /= p.sum() if normalize else np.exp(L[t] - L[t].max()).sum()
        # float32 logits of H = 128 terms below 6 in magnitude: a few 1e-5 in the exponent
        assert np.allclose(r["w"][t].cpu().numpy(), p, rtol=1e-4, atol=0)
    out = moe.forward_w8a8(x, w, q1, s1, q2, s2, k, normalize=normalize, router_bias=bias)
    p = moe.permute(r["idx"], E, hidden=x)
    assert moe.get_error(p["err_word"]) == (_abi.MOE_OK, 0)
    y = moe.expert_ffn_w8a8(p["x_perm"], p["offsets"], q1, s1, q2, s2)
    want = moe.combine(y, p["perm_dst"], r["w"], T, k)
    sure = r["near_tie"] == 0
    d = (out.double() - want.double()).abs()[sure]
    assert torch.all(d <= 1e-5 * k * float(y.float().abs().max()) + 2.0 ** -7 * want.double().abs()[sure])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_a_token_that_is_not_finite_comes_out_nan_alone(T, E, k, value):
    x, w, q1, s1, q2, s2 = inputs(T, E, 2)
    ws = torch.full((moe.w8a8_workspace_size(T, H, E, k, I),), 0x5A, dtype=torch.uint8, device="cuda")
    want = moe.forward_w8a8(x, w, q1, s1, q2, s2, k, workspace=ws)
    rows = sorted({3, T - 1})
    bad = x.clone()
    bad[rows, 11] = value
    if T > 100:
        bad[130 % T] = float("nan")       # every value, in another tile
        rows = sorted({3, 130 % T, T - 1})
    valid(moe.route(bad, w, k)["idx"], E)
    out = moe.forward_w8a8(bad, w, q1, s1, q2, s2, k, workspace=ws)
    assert moe.get_error(moe.workspace_error_word(ws)) == (_abi.MOE_OK, 0)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.isnan(out[rows].float()).all() and torch.equal(out[keep], want[keep])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_the_unquantised_layer_keeps_a_nan_in_its_token(T, E, k, dt):
    x, w, q1, s1, q2, s2 = inputs(T, E, 3)
    x, w = x.to(dt), w.to(dt)
    f1, f2 = (q1.float() * s1[:, :, None]).to(dt), (q2.float() * s2[:, :, None]).to(dt)
    want = moe.forward(x, w, f1, f2, k)
    bad = x.clone()
    bad[3, 11] = float("nan")
    out = moe.forward(bad, w, f1, f2, k)
    keep = torch.arange(T, device="cuda") != 3
    assert torch.isnan(out[3].float()).all() and torch.equal(out[keep], want[keep])
