"""int8 rows, products, FFN, layer and balance loss where offsets of elements pass 32 bits:
sampled rows against float64 of the same operator (bounds: w8a8_util, test_gpu_balance)."""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_15_b200 as moe
from w8a8_util import U32, UB, ffn_with_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def weights(g, *shape):
    q = torch.randint(-127, 128, shape, dtype=torch.int8, device="cuda", generator=g)
    s = (torch.rand(shape[:-1], device="cuda", generator=g) + 0.5) / 127 / shape[-1] ** 0.5
    return q, s


def some(rows, n=40):
    """The first and last rows and some between, rows around element 2^31 among them."""
    return torch.unique(torch.tensor([0, 1, rows - 2, rows - 1] + [int(r) for r in np.linspace(0, rows - 1, n)]))


def quantized(x):
    v = x.double()
    top = v.abs().amax(1)
    return (127 * v / top[:, None]).round(), (top.float() / torch.full_like(top, 127, dtype=torch.float32))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows(dt):
    rows, K = 300007, 8192
    x = torch.empty((rows, K), dtype=dt, device="cuda").normal_(generator=gen(1))
    q, s = moe.quantize_rows(x)
    at = some(rows).cuda()
    rq, rs = quantized(x[at])
    assert torch.equal(q[at].double(), rq) and torch.equal(s[at], rs)


@pytest.mark.parametrize("rows,N,E,dt", [(20011, 131104, 0, torch.bfloat16), (20011, 131104, 3, torch.float32),
                                         (9001, 262176, 256, torch.bfloat16), (3, (1 << 26) + 32, 0, torch.bfloat16)])
def test_products(rows, N, E, dt):
    """The kernels of many rows (dense, grouped) and of few rows per expert."""
    K, g = 16, gen(2)
    q = torch.randint(-127, 128, (rows, K), dtype=torch.int8, device="cuda", generator=g)
    s = torch.rand(rows, device="cuda", generator=g) + 0.5
    w, ws = weights(g, max(E, 1), N, K)
    cut = np.sort(np.random.default_rng(3).integers(0, rows + 1, max(E, 1) - 1))
    off = np.concatenate([[0], cut, [rows]]).astype(np.int32)
    if E:
        out = moe.matmul_q8(q, s, w, ws, offsets=torch.from_numpy(off).cuda(), out_dtype=dt)
    else:
        out = moe.matmul_q8(q, s, w[0], ws[0], out_dtype=dt)
    uout = UB if dt == torch.bfloat16 else U32
    for r in some(rows, 10 if N > 1 << 20 else 40).tolist():
        e = int(np.searchsorted(off[1:], r, side="right"))
        for a in range(0, N, 1 << 22):
            y = (w[e, a:a + (1 << 22)].double() @ q[r].double()) * s[r].double() * ws[e, a:a + (1 << 22)].double()
            d = (out[r, a:a + (1 << 22)].double() - y).abs()
            assert torch.all(d <= 1.01 * (3 * U32 + uout) * y.abs() + 1e-30), (r, a)


def test_ffn_of_many_rows_and_channels():
    rows, H, I, g = 70001, 32, 32768, gen(4)
    x = torch.randn((rows, H), device="cuda", generator=g).bfloat16()
    q1, s1 = weights(g, 1, 2 * I, H)
    q2, s2 = weights(g, 1, H, I)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    y = moe.expert_ffn_w8a8(x, off, q1, s1, q2, s2)
    at = some(rows, 12)
    h = [a[0].cpu().numpy() for a in (q1, s1, q2, s2)]
    ref, bound = ffn_with_bound(x[at.cuda()].cpu().double().numpy(), *h, "interleaved", (1.0, 0.0, float("inf")))
    assert np.all(np.abs(y[at.cuda()].cpu().double().numpy() - ref) <= bound)


def test_layer_of_many_tokens():
    """The permuted rows pass 2^31 elements: the same as the tokens in two halves."""
    T, H, E, k, I, g = 40000, 8192, 8, 8, 32, gen(5)
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    router = (torch.randn((E, H), device="cuda", generator=g) / 64).bfloat16()
    w = [*weights(g, E, 2 * I, H), *weights(g, E, H, I)]
    out = moe.forward_w8a8(x, router, *w, k)
    halves = torch.cat([moe.forward_w8a8(h.contiguous(), router, *w, k) for h in (x[:T // 2], x[T // 2:])])
    assert torch.equal(out, halves)


def test_balance():
    """Equal blocks of tokens: the counts of one block times their number, its probabilities,
    and the same gradient rows (scaled by a power of two) in every block."""
    n, E, k, times = 1 << 18, 256, 4, 64
    lg = torch.randn((n, E), device="cuda", generator=gen(6))
    idx = torch.topk(lg, k, 1).indices.int()
    one = moe.balance_loss(lg, idx)
    d1 = moe.balance_loss_backward(lg, k, one["counts"], one["tokens"])
    big = lg.expand(times, n, E).reshape(times * n, E)
    r = moe.balance_loss(big, idx.expand(times, n, k).reshape(times * n, k))
    assert torch.equal(r["counts"], one["counts"] * times) and int(r["tokens"]) == times * n
    p = torch.softmax(lg.double(), 1).mean(0)
    assert torch.all((r["probs"][0].double() - p).abs() <= 128 * U32 * p)
    d = moe.balance_loss_backward(big, k, r["counts"], r["tokens"])
    for b in (0, 31, 32, times - 1):
        assert torch.equal(d[b * n:(b + 1) * n] * times, d1)
