"""The balance loss on the GPU where its ranges, sequences and sums are at their worst:
offsets that decrease, blocks that walk many rows, very many tokens.  Bounds: test_gpu_balance."""
import numpy as np
import pytest
import torch

import mixture_experts_ffn_15_b200 as moe
from mixture_experts_ffn_15_b200 import _abi
from test_gpu_balance import compare, run

pytestmark = pytest.mark.gpu


def batch(T, E, k, seed):
    rng = np.random.default_rng(seed)
    lg = (rng.standard_normal((T, E)) * 2 + rng.standard_normal(E)).astype(np.float32).astype(np.float64)
    return lg, np.argsort(-lg, axis=1, kind="stable")[:, :k], rng


def poisoned(T, E, S):
    n = moe.load_library().moe_balance_loss_workspace_size(T, E, S)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("T,seqs", [
    (40, [[0, 20, 10, 40], [5, 40], [30, 10, 40], [0, 50], [-5, 40], [40, 0], [90, 95, 100], [40, 40, 3]]),
    (1000, [[0, 600, 300, 700, 650, 1000], [700, 100, 900, 200, 1000], [0, 5000, 20, 30], [300, 1000, 0, 1000],
            [1000, 0, 0, 0], [0, 64, 128, 64, 64, 192, 128, 900], [-7, 63, -8, 65, 2000], [999, 1000, 1000, 5]]),
    (12000, [[0, 9000, 30, 9001, 11000, 200, 12000], [11999, 12000, 1], [0] + [7000, 100] * 600 + [12000]])])
def test_offsets_that_decrease_make_empty_sequences(T, seqs):
    """The offsets count as their running maximum, clamped to the batch; never-written memory
    has no part in the results; the error word tells."""
    lg, idx, rng = batch(T, 12, 2, T)
    mask = rng.random(T) < 0.8
    for seq in seqs:
        bounds = np.maximum.accumulate(np.clip(seq, 0, T))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run(lg, idx, 0.5, mask, seq, err_word=err, workspace=poisoned(T, 12, len(seq) - 1))
        compare(got, lg, idx, 0.5, mask, bounds)
        assert moe.get_error(err) == (_abi.MOE_ERR_DEVICE, 1), seq


@pytest.mark.parametrize("T,S", [(1, 3000), (700, 2500), (3000, 3000), (40000, 1500), (0, 5)])
def test_many_sequences(T, S):
    """More sequences than a block has threads, most of them empty or of a few tokens."""
    lg, idx, rng = batch(T, 8, 2, S)
    seq = np.concatenate([[0], np.sort(rng.integers(0, T + 1, S - 1)), [T]])
    if T == 700:
        seq = np.minimum(np.arange(S + 1) // 3, T)   # empty ones between all the others
        seq[-1] = T
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(lg, idx, 1.0, None, seq, err_word=err, workspace=poisoned(T, 8, S))
    compare(got, lg, idx, 1.0, None, seq)
    assert moe.get_error(err) == (_abi.MOE_OK, 0)


def test_probabilities_of_very_many_tokens():
    """Every row the same, its probabilities such that each float32 addition of a long sum
    rounds the same way (1000 of them in a row: 230 U32 off).  Bound: (18 + 2.3 |logit - max|)
    U32 of a probability, 31 + 32 additions of a lane, 5 of the lanes, 31 of the warps, the
    result's rounding: 119 U32."""
    T, E, x = 148 * 32 * 1000 + 5, 160, 0.101
    row = torch.zeros(E, dtype=torch.float32, device="cuda")
    row[7] = x
    logits = row.expand(T, E).contiguous()
    idx = torch.arange(T, dtype=torch.int32, device="cuda").remainder(E)[:, None].contiguous()
    r = moe.balance_loss(logits, idx, coef=1.0)
    p = torch.softmax(row.double(), 0)
    U32 = 2.0 ** -24
    assert torch.all((r["probs"][0].double() - p).abs() <= 119 * U32 * p)
    assert torch.equal(r["counts"][0].long(), torch.bincount(idx[:, 0], minlength=E))
    loss = float(E * (r["counts"][0].double() / T * p).sum())
    assert abs(float(r["loss"]) - loss) <= 121 * U32 * loss      # its sum in float64, one rounding
    d = moe.balance_loss_backward(logits, 1, r["counts"], r["tokens"])
    assert torch.equal(d, d[:1].expand(T, E))                   # equal rows, equal bits


@pytest.mark.parametrize("E", [1, 8, 9, 60, 130])
def test_long_ranges(E):
    """T where a lane folds its sums several times, for each number of lanes; with E = 130, T
    where a block's range passes its largest number of rows.  Bound: (18 + 2.3 |logit - max|)
    U32 with the maximum at most 9 above, 31 + 16 + 5 + 31 additions, one rounding: 123 U32."""
    lanes = 1
    while lanes * 8 < E:
        lanes *= 2
    T = 148 * 32 * (1024 if E > 60 else 65) * (32 // lanes) + 3
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn((T, E), generator=g, device="cuda")
    mask = torch.rand((T,), generator=g, device="cuda") < 0.9
    seq = torch.tensor([0, T // 3, T // 3, T - 1], dtype=torch.int32, device="cuda")
    idx = logits.argmax(1, keepdim=True).int()
    r = moe.balance_loss(logits, idx, mask=mask, seq_offsets=seq)
    p = torch.softmax(logits.double(), 1)
    for s in range(3):
        a, z = int(seq[s]), int(seq[s + 1])
        m = mask[a:z]
        n = int(m.sum())
        assert int(r["tokens"][s]) == n
        assert torch.equal(r["counts"][s].long(), torch.bincount(idx[a:z, 0][m], minlength=E))
        want = p[a:z][m].sum(0) / max(n, 1)
        assert torch.all((r["probs"][s].double() - want).abs() <= 128 * 2.0 ** -24 * want)


def reference(lg, idx, k, coef, mask, seq):
    """loss, counts, probs, dlogits and the gradient's bound in float64, whole tensors at a time."""
    T, E = lg.shape
    p = torch.softmax(lg.double(), 1)
    bounds = torch.tensor([0, T] if seq is None else list(seq), device="cuda")
    S = bounds.numel() - 1
    sid = torch.searchsorted(bounds[1:].contiguous(), torch.arange(T, device="cuda"), right=True).clamp_max(S - 1)
    live = (torch.arange(T, device="cuda") < bounds[-1]) & (torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask)
    n = torch.zeros(S, dtype=torch.long, device="cuda").index_add_(0, sid, live.long())
    flat = (sid[:, None] * E + idx.long())[live].reshape(-1)
    counts = torch.bincount(flat, minlength=S * E).view(S, E)
    probs = torch.zeros((S, E), dtype=torch.float64, device="cuda").index_add_(0, sid, p * live[:, None])
    nd = n.clamp_min(1).double()
    probs = probs / nd[:, None]
    f = counts / (nd[:, None] * k)
    f0 = torch.where(n[:, None] > 0, f - 1.0 / E, 0.0)[sid]
    dot, mag = (p * f0).sum(1, keepdim=True), (p * f0.abs()).sum(1, keepdim=True)
    scale = (coef * E / (S * nd))[sid][:, None] * live[:, None]
    # the bound of test_gpu_balance, the reference's own rounding from f - 1/E instead of f
    own = (E + 4) * 2.0 ** -53 * f.amax(1)[sid][:, None]
    bound = scale * p * (160 * 2.0 ** -24 * ((f0 - dot).abs() + mag) + own) + 1e-37
    return coef / S * E * (f * probs).sum(), counts, probs, n, scale * p * (f0 - dot), bound


@pytest.mark.parametrize("E", [256, 255, 128, 97, 12])
@pytest.mark.parametrize("S", [0, 1, 20, 700])
@pytest.mark.parametrize("masked", [False, True])
def test_blocks_of_many_rows(E, S, masked):
    """Up to 13 rows a lane forward and 17 backward, two of them loaded ahead, with sequence
    bounds inside the blocks and a tail that belongs to no sequence."""
    T, k = 60013, min(8, E)
    g = torch.Generator(device="cuda").manual_seed(E + S)
    lg = torch.randn((T, E), generator=g, device="cuda") * 1.5 + torch.randn(E, generator=g, device="cuda")
    idx = torch.topk(lg, k, 1).indices.int()
    mask = torch.rand(T, generator=g, device="cuda") < 0.7 if masked else None
    seq = None
    if S:
        rng = np.random.default_rng(S)
        seq = np.concatenate([[0], np.sort(rng.integers(0, T + 1, S - 1)), [T - 11]])
        seq = np.minimum(seq, T - 11)
    s = None if seq is None else torch.from_numpy(seq.astype(np.int32)).cuda()
    r = moe.balance_loss(lg, idx, coef=0.01, mask=mask, seq_offsets=s)
    d = moe.balance_loss_backward(lg, k, r["counts"], r["tokens"], coef=0.01, mask=mask, seq_offsets=s)
    loss, counts, probs, n, grad, bound = reference(lg, idx, k, 0.01, mask, seq)
    assert torch.equal(r["counts"].long(), counts) and torch.equal(r["tokens"].long(), n)
    U32 = 2.0 ** -24
    assert torch.all((r["probs"].double() - probs).abs() <= 128 * U32 * probs + 1e-37)
    assert abs(float(r["loss"]) - float(loss)) <= 132 * U32 * float(loss)
    over = (d.double() - grad).abs() - bound
    assert torch.all(over <= 0), (float(over.max()), int(over.argmax()) // E)
    again = moe.balance_loss(lg, idx, coef=0.01, mask=mask, seq_offsets=s)
    assert all(torch.equal(again[a], r[a]) for a in r)


@pytest.mark.parametrize("T", [90, 1500])
def test_long_runs_of_empty_sequences_between_others(T):
    """Runs of 15 to 1100 empty sequences inside a block, at its ends and at the batch's, some
    of them by offsets that decrease."""
    lg, idx, rng = batch(T, 8, 2, T)
    seq = [0] * 17
    for at, times in ((3, 15), (4, 16), (64, 33), (66, 1100), (min(T - 5, 512), 31), (T - 2, 40), (T, 20)):
        seq += [at] * times
    for s in (seq, [v - (i % 7 == 3) * min(v, 2) for i, v in enumerate(seq)]):
        bounds = np.maximum.accumulate(np.clip(s, 0, T))
        got = run(lg, idx, 1.0, None, s, workspace=poisoned(T, 8, len(s) - 1))
        compare(got, lg, idx, 1.0, None, bounds)
