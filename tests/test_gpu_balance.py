"""The balance loss, its counts and its gradient on the GPU against float64.

Bounds, with U32 = 2^-24: the difference logit - max rounds once, its product with log2 e once,
log2 e itself is off by less than 0.3 U32: 2.3 |logit - max| U32 in the exponent; the
exponential is within 2 ulp (4 U32), the sum of E terms by a tree of depth 5 on up to 8 terms
a lane rounds 12 times, the quotient and the product once each: (18 + 2.3 |logit - max|) U32.
Logits here stay within 20 of their row's maximum: 64 U32 relative.
P adds float32 sums of at most 27 such terms a lane, over 5 shuffles and 32 warps: another
64 U32 (the blocks' sums are added in float64).
The loss is a sum of non-negative terms f P: the same relative bound, and its own rounding.
The gradient coef E / (S n) p (f - sum f p), with f less 1/E: |d| <= 64 U32 p |f - dot| from
p, and (64 + 16) U32 sum p |f| from the dot product; f, the scale and the products a few U32
more: 160 U32 scale p (|f - dot| + sum p |f|) covers them."""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_15_b200 as moe
from mixture_experts_ffn_15_b200 import _abi
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def softmax(L):
    with np.errstate(invalid="ignore"):
        m = L.max(1, keepdims=True)
        p = np.exp(L - np.where(np.isfinite(m), m, 0.0))
        s = p.sum(1, keepdims=True)
        return p / np.where(s > 0, s, 1.0)


def grad_bound(lg, ref, k, coef, mask, seq):
    T, E = lg.shape
    p = softmax(lg)
    seq = [0, T] if seq is None else list(seq)
    S = len(seq) - 1
    out = np.zeros((T, E))
    for s in range(S):
        n = ref["tokens"][s]
        if n == 0:
            continue
        f = ref["counts"][s] / (n * k) - 1.0 / E
        for t in range(seq[s], seq[s + 1]):
            dot, mag = np.sum(p[t] * f), np.sum(p[t] * np.abs(f))
            own = (E + 4) * 2.0 ** -53 * np.max(ref["counts"][s] / (n * k))   # the reference's rounding
            out[t] = coef * E / (S * n) * p[t] * (160 * U32 * (np.abs(f - dot) + mag) + own)
    return out + 1e-37


def run(lg, idx, coef=1.0, mask=None, seq=None, **kw):
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
    L, m, s = dev(lg.astype(np.float32)), dev(mask), dev(None if seq is None else np.asarray(seq, dtype=np.int32))
    i = dev(idx.astype(np.int32))
    r = moe.balance_loss(L, i, coef=coef, mask=m, seq_offsets=s, **kw)
    d = moe.balance_loss_backward(L, idx.shape[1], r["counts"], r["tokens"], coef=coef, mask=m, seq_offsets=s)
    return {k: v.cpu().numpy() for k, v in dict(r, dlogits=d).items()}


def compare(got, lg, idx, coef, mask, seq):
    ref = O.balance_loss(lg, idx, coef, mask, seq)
    assert np.array_equal(got["counts"], ref["counts"]) and np.array_equal(got["tokens"], ref["tokens"])
    assert np.all(np.abs(got["probs"] - ref["probs"]) <= 128 * U32 * ref["probs"] + 1e-37)
    assert abs(got["loss"][0] - ref["loss"]) <= 132 * U32 * abs(ref["loss"])
    b = grad_bound(lg, ref, idx.shape[1], abs(coef), mask, seq)
    d = np.abs(got["dlogits"] - ref["dlogits"])
    assert np.all(d <= b), (np.max(d - b), np.unravel_index(np.argmax(d - b), d.shape))


CASES = [  # T, E, k, S (0: no seq_offsets), masked share
    (1, 1, 1, 0, 0.0), (1, 8, 2, 0, 0.0), (3, 5, 5, 0, 0.0), (64, 8, 2, 0, 0.0), (65, 33, 3, 0, 0.3),
    (200, 128, 8, 0, 0.0), (1000, 60, 4, 3, 0.2), (777, 256, 8, 1, 0.5), (130, 100, 7, 40, 0.1),
    (4099, 64, 4, 5, 0.1), (20001, 16, 2, 0, 0.0), (50, 255, 1, 2, 0.9),
]


@pytest.mark.parametrize("T,E,k,S,masked", CASES)
def test_balance_loss_and_gradient(T, E, k, S, masked):
    rng = np.random.default_rng(T + E)
    lg = (rng.standard_normal((T, E)) * 2 + rng.standard_normal(E)).astype(np.float32).astype(np.float64)
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :k]
    mask = rng.random(T) >= masked if masked else None
    seq = np.concatenate([[0], np.sort(rng.integers(0, T + 1, S - 1)), [T]]) if S else None
    compare(run(lg, idx, 0.01, mask, seq), lg, idx, 0.01, mask, seq)


def test_sequences_that_are_empty_short_and_leave_a_tail():
    rng = np.random.default_rng(1)
    T, E, k = 500, 32, 2
    lg = rng.standard_normal((T, E)).astype(np.float32).astype(np.float64)
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :k]
    for seq in ([0, 0, 1, 1, 3, 300, 300, 450], [0, 0, 0], [0, 500, 500], [0, 64, 128, 129, 500], [0, 0], [0, 7]):
        mask = rng.random(T) < 0.7
        mask[1:3] = False          # a whole sequence masked in the first list
        compare(run(lg, idx, 1.5, mask, seq), lg, idx, 1.5, mask, seq)


def test_one_short_sequence_in_a_small_batch():
    rng = np.random.default_rng(8)
    lg = rng.standard_normal((20, 16)).astype(np.float32).astype(np.float64)
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :2]
    for seq in ([0, 0], [0, 3], [0, 20], [0, 0, 20], [0, 20, 20]):
        compare(run(lg, idx, 1.0, seq=seq), lg, idx, 1.0, None, seq)


def test_no_tokens_at_all():
    lg, idx = np.zeros((0, 8)), np.zeros((0, 2), dtype=np.int64)
    r = run(lg, idx)
    assert r["loss"][0] == 0 and not r["counts"].any() and not r["probs"].any() and r["tokens"].tolist() == [0]
    r = run(np.zeros((5, 8)), np.zeros((5, 2), dtype=np.int64), mask=np.zeros(5, dtype=bool))
    assert r["loss"][0] == 0 and not r["counts"].any() and not r["dlogits"].any()


def test_the_same_id_twice_and_ids_out_of_range():
    lg = np.random.default_rng(2).standard_normal((40, 8)).astype(np.float32).astype(np.float64)
    idx = np.zeros((40, 3), dtype=np.int64)
    idx[:, 1:] = 5                                       # twice in every token
    compare(run(lg, idx, 1.0), lg, idx, 1.0, None, None)
    idx[7, 0], idx[9, 2] = -1, 8
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    compare(run(lg, idx, 1.0, err_word=err), lg, idx, 1.0, None, None)
    assert moe.get_error(err) == (_abi.MOE_ERR_DEVICE, 1)


def test_bad_sequence_offsets_are_reported():
    lg, idx = np.zeros((40, 8)), np.zeros((40, 2), dtype=np.int64)
    for seq in ([0, 50], [1, 40], [0, 20, 10, 40], [-5, 40]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        run(lg, idx, seq=seq, err_word=err)
        assert moe.get_error(err) == (_abi.MOE_ERR_DEVICE, 1), seq


def test_infinite_and_nan_logits():
    rng = np.random.default_rng(3)
    lg = rng.standard_normal((30, 16)).astype(np.float32).astype(np.float64)
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :2]
    lg[4, 3:] = -np.inf                   # experts masked out
    lg[5] = -np.inf                       # nothing left
    lg[6] = np.finfo(np.float32).min      # the type's lowest value everywhere: uniform
    got = run(lg, idx, 1.0)
    assert not got["dlogits"][5].any() and not got["dlogits"][4, 3:].any()
    compare(got, lg, idx, 1.0, None, None)
    # NaN in masked places has no effect, in a valid token it shows
    bad = lg.copy()
    bad[9, 2], bad[10] = np.nan, np.inf
    mask = np.ones(30, dtype=bool)
    mask[9:11] = False
    a, b = run(bad, idx, 1.0, mask), run(lg, idx, 1.0, mask)
    for n in a:
        assert np.array_equal(a[n], b[n]), n
    r = run(bad, idx, 1.0)
    assert np.isnan(r["loss"][0]) and np.isnan(r["dlogits"][9]).all() and np.isnan(r["dlogits"][10]).all()
    assert np.isfinite(r["dlogits"][11]).all() and np.array_equal(r["counts"], b["counts"]) is False


def test_gradient_by_differences_and_upstream_gradient():
    """Central differences of the GPU's loss along random directions: the loss has float32
    resolution (2^-24 of ~1), so a step of 2^-6 gives slopes to about 2^-17, and the
    third derivative adds step^2 / 6 of the direction's cube, below 1e-4 here."""
    rng = np.random.default_rng(4)
    T, E, k = 16, 8, 2
    lg = rng.standard_normal((T, E)).astype(np.float32).astype(np.float64)
    idx = np.argsort(-lg, axis=1, kind="stable")[:, :k]
    g = run(lg, idx)["dlogits"].astype(np.float64)
    for _ in range(5):
        v = np.sign(rng.standard_normal((T, E)))
        h = 2.0 ** -6
        num = (float(run(lg + h * v, idx)["loss"][0]) - float(run(lg - h * v, idx)["loss"][0])) / (2 * h)
        assert abs(num - np.sum(g * v)) < 2.0 ** -16 + 1e-4
    L = torch.from_numpy(lg.astype(np.float32)).cuda()
    i = torch.from_numpy(idx.astype(np.int32)).cuda()
    r = moe.balance_loss(L, i, coef=0.5)
    one = moe.balance_loss_backward(L, k, r["counts"], r["tokens"], coef=0.5)
    up = torch.tensor([-4.0], device="cuda")
    four = moe.balance_loss_backward(L, k, r["counts"], r["tokens"], coef=0.5, grad_loss=up)
    assert torch.equal(four, one * -4)


def test_after_route_the_same_bits_and_captured():
    """route -> balance_loss -> backward as a training step calls them: repeated calls give
    the same bits, also captured in a graph, on another stream and with a kept workspace."""
    T, H, E, k = 300, 128, 64, 4
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    w = (torch.randn((E, H), generator=g, device="cuda") * 0.1).bfloat16()
    r = moe.route(x, w, k)
    lib = moe.load_library()
    ws = torch.full((lib.moe_balance_loss_workspace_size(T, E, 1),), 0xFF, dtype=torch.uint8, device="cuda")

    def step(stream=None):
        b = moe.balance_loss(r["logits"], r["idx"], coef=0.01, workspace=ws, stream=stream)
        d = moe.balance_loss_backward(r["logits"], k, b["counts"], b["tokens"], coef=0.01, stream=stream)
        return b, d
    b0, d0 = step()
    L = r["logits"].cpu().numpy().astype(np.float64)
    compare({k_: v.cpu().numpy() for k_, v in dict(b0, dlogits=d0).items()}, L, r["idx"].cpu().numpy(), 0.01, None, None)
    counts = moe.permute(r["idx"], E)["counts"]
    assert torch.equal(b0["counts"][0], counts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b1, d1 = step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b2, d2 = step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for b, d in ((b1, d1), (b2, d2)):
        assert torch.equal(d, d0) and all(torch.equal(b[n], b0[n]) for n in b0)


def test_binding_refuses_mismatches():
    L = torch.zeros(8, 4, device="cuda")
    i = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        moe.balance_loss(L.half(), i)
    with pytest.raises(TypeError):
        moe.balance_loss(L, i.long())
    with pytest.raises(ValueError):
        moe.balance_loss(L, i[:7])
    with pytest.raises(ValueError):
        moe.balance_loss(L, i, mask=torch.ones(7, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        moe.balance_loss(L, i, seq_offsets=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(moe.MoEError):
        moe.balance_loss(L, torch.zeros(8, 5, dtype=torch.int32, device="cuda"))   # k > E
    with pytest.raises(ValueError):
        moe.balance_loss_backward(L, 2, i, i)
