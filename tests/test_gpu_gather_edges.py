"""The layer's gather of token rows at row lengths that leave lanes of a warp without elements."""
import pytest
import torch

import mixture_experts_ffn_15_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,H,I,dt", [
    (130, 256, 30, 128, 64, torch.bfloat16), (130, 64, 32, 128, 64, torch.bfloat16),
    (300, 128, 20, 128, 64, torch.bfloat16), (600, 60, 20, 128, 64, torch.bfloat16),
    (20000, 64, 17, 64, 64, torch.bfloat16), (3000, 64, 24, 2112, 64, torch.bfloat16),
    (3000, 64, 9, 2176, 64, torch.bfloat16), (600, 40, 31, 8, 16, torch.float32), (700, 33, 20, 72, 24, torch.float32)])
def test_the_layer_equals_its_steps(T, E, k, H, I, dt):
    """More choices a token than lanes with elements of its row (in the last 4 KB of it): the
    destinations come from all lanes.  Layer and steps run the same kernels but for the gather."""
    g = torch.Generator(device="cuda").manual_seed(T + H)
    x = torch.randn((T, H), generator=g, device="cuda").to(dt)
    w = (torch.randn((E, H), generator=g, device="cuda") / H ** 0.5).to(dt)
    f1 = (torch.randn((E, 2 * I, H), generator=g, device="cuda") / H ** 0.5).to(dt)
    f2 = (torch.randn((E, H, I), generator=g, device="cuda") / I ** 0.5).to(dt)
    r = moe.route(x, w, k)
    p = moe.permute(r["idx"], E, hidden=x)
    want = moe.combine(moe.expert_ffn(p["x_perm"], p["offsets"], f1, f2), p["perm_dst"], r["w"], T, k)
    for _ in range(3):
        assert torch.equal(moe.forward(x, w, f1, f2, k), want)
