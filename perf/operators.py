"""Performance cases of the int8 expert products and of the router's balance loss.

Three operators, each in a plain form (elementary torch operations) and as the calls a
user of the framework makes:

  product   out = (round8(x) w_q^T) * x_scale[token] * w_scale[channel] (+ bias): int8 rows
            made from float rows (one scale a token), times int8 weights (one scale an
            output channel), dense or grouped by expert
  ffn       the grouped expert FFN on that product: fc1, SwiGLU, int8 rows again, fc2
  balance   the load-balance loss of the routing, its per-expert counts, and its gradient
            with respect to the router logits

`own` selects which of the two `run` does.
"""
import math

import numpy as np
import torch

own = False

INF = float("inf")
GPT_OSS = (1.702, 1.0, 7.0)
STANDARD = (1.0, 0.0, INF)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token through a dense projection: latency and one pass over the weights
        dict(name="product_one_token", op="product", rows=1, K=2816, N=1408, E=0, dt="bf16", bias=False, skew=0.0),
        # a small odd batch in float32 with a bias
        dict(name="product_61_rows_f32", op="product", rows=61, K=704, N=2816, E=0, dt="f32", bias=True, skew=0.0),
        # fc1's product of a batched decode step: 2048 routed rows, uneven experts, some empty
        dict(name="product_grouped_2048", op="product", rows=2048, K=2816, N=1408, E=128, dt="bf16", bias=False, skew=1.0),
        # a dense projection over a long odd prompt: compute bound
        dict(name="product_8191_rows", op="product", rows=8191, K=4096, N=4096, E=0, dt="bf16", bias=True, skew=0.0),
        # the expert FFN of a decode step of 4 tokens with 8 experts each
        dict(name="ffn_decode_32_rows", op="ffn", rows=32, H=2816, I=704, E=128, dt="bf16", layout="interleaved", bias=False, act="standard", skew=0.0),
        # a layer of test size
        dict(name="ffn_small_128_rows", op="ffn", rows=128, H=256, I=128, E=8, dt="bf16", layout="interleaved", bias=True, act="standard", skew=0.5),
        # batched decode: 256 tokens x 8, uneven experts, chunked fc1, biases, clipped SwiGLU
        dict(name="ffn_batched_2048_rows", op="ffn", rows=2048, H=2816, I=704, E=128, dt="bf16", layout="chunked", bias=True, act="gpt_oss", skew=1.0),
        # prefill: 8192 tokens x 8
        dict(name="ffn_prefill_65536_rows", op="ffn", rows=65536, H=2816, I=704, E=128, dt="bf16", layout="chunked", bias=False, act="standard", skew=0.25),
        # the router of a small layer
        dict(name="balance_64_tokens", op="balance", T=64, E=8, k=2, S=1, masked=0.0),
        # a training micro-batch as one group of tokens
        dict(name="balance_8192_tokens", op="balance", T=8192, E=128, k=8, S=1, masked=0.0),
        # a padded batch of sequences of uneven lengths, the loss taken sequence by sequence
        dict(name="balance_32768_ragged", op="balance", T=32768, E=64, k=4, S=9, masked=0.1),
        # a large batch over many experts, odd length
        dict(name="balance_131071_tokens", op="balance", T=131071, E=256, k=8, S=1, masked=0.05),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "ffn", "balance"])
    if op == "balance":
        E = rng.choice([8, 16, 60, 64, 96, 128, 160, 256])
        return dict(op=op, T=_log_uniform(rng, 1, 131071), E=E, k=rng.randint(1, 8),
                    S=rng.choice([1, 1, rng.randint(2, 64)]), masked=rng.choice([0.0, rng.uniform(0.0, 0.5)]))
    bias = rng.random() < 0.5
    if op == "product":
        E = rng.choice([0, 0, _log_uniform(rng, 2, 128)])
        most = 88 if E else 128          # grouped weights stay below the largest listed case's
        return dict(op=op, rows=_log_uniform(rng, 1, 8191), K=16 * _log_uniform(rng, 4, 2 * most),
                    N=32 * _log_uniform(rng, 2, most // 2 if E else most), E=E,
                    dt=rng.choice(["bf16", "bf16", "f32"]), bias=bias, skew=rng.uniform(0.0, 1.0))
    E = _log_uniform(rng, 2, 128)
    H = 32 * _log_uniform(rng, 4, 88)
    inter = 32 * _log_uniform(rng, 2, 22)
    return dict(op=op, rows=_log_uniform(rng, 1, 8192), H=H, I=inter, E=E, dt="bf16",
                layout=rng.choice(["interleaved", "chunked"]), bias=bias,
                act=rng.choice(["standard", "gpt_oss"]), skew=rng.uniform(0.0, 1.0))


def _used(rows, E):
    """Experts that `rows` rows reach on average."""
    return E * (1.0 - (1.0 - 1.0 / E) ** rows)


def work(case):
    c = case
    if c["op"] == "balance":
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        # logits read by either pass of one kernel each, ids, mask; gradient and sums written
        return {"bytes": 2 * 4 * T * E + 4 * T * E + 4 * T * k + 2 * T + 8 * S * E, "flops": 12.0 * T * E}
    es = 2 if c["dt"] == "bf16" else 4
    rows = c["rows"]
    if c["op"] == "product":
        K, N, E = c["K"], c["N"], c["E"]
        u = _used(rows, E) if E else 1
        return {"bytes": rows * K * es + u * N * (K + 4) + rows * N * es + 4 * rows, "flops": 2.0 * rows * K * N}
    H, inter = c["H"], c["I"]
    u = _used(rows, c["E"])
    return {"bytes": 2 * rows * H * es + u * (3 * inter * H + 4 * (2 * inter + H)),
            "flops": 2.0 * rows * 3 * inter * H}


# ------------------------------------------------------------------------------ inputs

def _sizes(rows, E, skew, rng):
    p = np.exp(skew * rng.standard_normal(E))
    return rng.multinomial(rows, p / p.sum())


def _weights(g, *shape):
    """int8 weight rows and their float32 scales: q * scale is about N(0, 1 / in_features)."""
    q = (torch.randn(shape, generator=g, device=DEV) * (127 / 4)).round_().clamp_(-127, 127).to(torch.int8)
    s = (torch.rand(shape[:-1], generator=g, device=DEV) * 0.5 + 0.75) * (4 / 127) / math.sqrt(shape[-1])
    return q, s


def _grouping(c, seed, st):
    E, rows = c["E"], c["rows"]
    n = _sizes(rows, E, c["skew"], np.random.default_rng([seed, 77]))
    off = np.concatenate([[0], np.cumsum(n)])
    st["offsets"] = torch.from_numpy(off.astype(np.int32)).to(DEV)
    st["cap"] = int(n.max())      # the host's plan of the plain form: rows of the fullest expert


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": c}
    if c["op"] == "balance":
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        lg = torch.randn((T, E), generator=g, device=DEV) * 1.06
        lg += torch.randn((E,), generator=g, device=DEV) * 0.5
        st["logits"] = lg
        st["idx"] = torch.topk(lg, k, dim=1).indices.to(torch.int32)
        rng = np.random.default_rng([seed, 78])
        st["mask"] = st["seq"] = None
        if S > 1:
            cut = np.sort(rng.integers(0, T + 1, S - 1))
            st["seq"] = torch.from_numpy(np.concatenate([[0], cut, [T]]).astype(np.int32)).to(DEV)
        if c["masked"] > 0:
            st["mask"] = torch.rand((T,), generator=g, device=DEV) >= c["masked"]
        st["coef"] = 0.01
        return st
    dt = DT[c["dt"]]
    rows = c["rows"]
    if c["op"] == "product":
        K, N, E = c["K"], c["N"], c["E"]
        st["x"] = torch.randn((rows, K), generator=g, device=DEV).to(dt)
        shape = (E, N, K) if E else (N, K)
        st["w"], st["ws"] = _weights(g, *shape)
        st["bias"] = (torch.randn(shape[:-1], generator=g, device=DEV) * 0.5).to(dt) if c["bias"] else None
        st["out"] = torch.zeros((rows, N), dtype=dt, device=DEV)
        st["offsets"], st["cap"] = None, rows
        if E:
            _grouping(c, seed, st)
        return st
    H, inter, E = c["H"], c["I"], c["E"]
    st["x"] = torch.randn((rows, H), generator=g, device=DEV).to(dt)
    st["w1"], st["s1"] = _weights(g, E, 2 * inter, H)
    st["w2"], st["s2"] = _weights(g, E, H, inter)
    st["b1"] = (torch.randn((E, 2 * inter), generator=g, device=DEV) * 0.5).to(dt) if c["bias"] else None
    st["b2"] = (torch.randn((E, H), generator=g, device=DEV) * 0.5).to(dt) if c["bias"] else None
    st["out"] = torch.zeros((rows, H), dtype=dt, device=DEV)
    st["swiglu"] = GPT_OSS if c["act"] == "gpt_oss" else STANDARD
    _grouping(c, seed, st)
    if own:
        import mixture_experts_ffn_15_b200 as moe
        st["workspace"] = moe.alloc_workspace(moe.expert_ffn_w8a8_workspace_size(rows, H, E, inter), DEV)
    return st


# -------------------------------------------------------------------------- plain form

def _round8(x):
    """x [rows, K] -> (whole numbers in [-127, 127] as float32, float32 scales [rows]); the
    quotient in 64 bits, since values next to a half decide which whole number they give."""
    amax = x.float().abs().amax(1)
    scale = amax / 127
    d = x.double() * 127 / amax.double().clamp_min(1e-300)[:, None]
    return d.round().float(), scale


def _grouped(q, w, offsets, cap):
    """Sums over k of q[r] * w[e of r] for every row: rows laid out as [E, cap, K], one
    batched product, and back."""
    E = w.shape[0]
    lo, hi = offsets[:-1].long(), offsets[1:].long()
    pos = lo[:, None] + torch.arange(cap, device=q.device)[None, :]
    inside = pos < hi[:, None]
    pad = q[torch.where(inside, pos, 0)] * inside[:, :, None]
    y = torch.bmm(pad, w.float().transpose(1, 2))
    out = torch.zeros((q.shape[0], w.shape[1]), dtype=torch.float32, device=q.device)
    out[pos[inside]] = y[inside]
    return out


def _expert_of(offsets, rows):
    return torch.searchsorted(offsets[1:].contiguous(), torch.arange(rows, device=offsets.device, dtype=torch.int32),
                              right=True)


def _swiglu(g, u, attr):
    alpha, beta, limit = attr
    g = g.clamp(max=limit)
    u = u.clamp(min=-limit, max=limit)
    return (u + beta) * g / (1 + torch.exp(-alpha * g))


def _plain_product(st):
    x, w = st["x"], st["w"]
    q, s = _round8(x)
    if st["offsets"] is None:
        y = (q @ w.float().t()) * s[:, None] * st["ws"][None, :]
        if st["bias"] is not None:
            y = y + st["bias"].float()
    else:
        e = _expert_of(st["offsets"], x.shape[0])
        y = _grouped(q, w, st["offsets"], st["cap"]) * s[:, None] * st["ws"][e]
        if st["bias"] is not None:
            y = y + st["bias"].float()[e]
    return {"out": y.to(x.dtype), "scale": s}


def _plain_ffn(st):
    x, off, cap = st["x"], st["offsets"], st["cap"]
    e = _expert_of(off, x.shape[0])
    q, s = _round8(x)
    h = _grouped(q, st["w1"], off, cap) * s[:, None] * st["s1"][e]
    if st["b1"] is not None:
        h = h + st["b1"].float()[e]
    inter = st["case"]["I"]
    gate, up = (h[:, :inter], h[:, inter:]) if st["case"]["layout"] == "chunked" else (h[:, 0::2], h[:, 1::2])
    a = _swiglu(gate, up, st["swiglu"])
    q, s = _round8(a)
    y = _grouped(q, st["w2"], off, cap) * s[:, None] * st["s2"][e]
    if st["b2"] is not None:
        y = y + st["b2"].float()[e]
    return y.to(x.dtype)


def _plain_balance(st):
    lg, idx, mask, seq, coef = st["logits"], st["idx"], st["mask"], st["seq"], st["coef"]
    T, E = lg.shape
    k = idx.shape[1]
    S = 1 if seq is None else seq.numel() - 1
    if seq is None:
        sid = torch.zeros((T,), dtype=torch.long, device=lg.device)
    else:
        sid = _expert_of(seq, T)
    valid = torch.ones((T,), dtype=torch.bool, device=lg.device) if mask is None else mask
    ex = torch.exp(lg - lg.amax(1, keepdim=True))
    p = ex / ex.sum(1, keepdim=True)
    pv = p * valid[:, None]
    tokens = torch.zeros((S,), dtype=torch.int32, device=lg.device).index_add_(0, sid, valid.to(torch.int32))
    hits = valid[:, None].expand(T, k).to(torch.int32)
    counts = torch.zeros((S * E,), dtype=torch.int32, device=lg.device)
    counts = counts.index_add_(0, (sid[:, None] * E + idx).reshape(-1), hits.reshape(-1)).reshape(S, E)
    # long sums in 64 bits
    sums = torch.zeros((S, E), dtype=torch.float64, device=lg.device).index_add_(0, sid, pv.double())
    n = tokens.clamp_min(1).double()
    probs = sums / n[:, None]
    # shares less their mean: sum_j p_j = 1, so the gradient does not change and loses less
    f = counts.double() / (n[:, None] * k)
    loss = (coef / S) * E * (f * probs).sum()
    f0 = torch.where(tokens[:, None] > 0, f - 1.0 / E, 0.0)
    scale = coef * E / S / n
    f0, scale = f0.float(), scale.float()
    ft = f0[sid]
    d = pv * (ft - (ft * p).sum(1, keepdim=True)) * scale[sid][:, None]
    return {"loss": loss.float().reshape(1), "counts": counts, "probs": probs.float(), "tokens": tokens, "dlogits": d}


# ---------------------------------------------------------------------- the user's calls

def _own(st):
    import mixture_experts_ffn_15_b200 as moe
    c = st["case"]
    if c["op"] == "product":
        q, s = moe.quantize_rows(st["x"])
        out = moe.matmul_q8(q, s, st["w"], st["ws"], offsets=st["offsets"], bias=st["bias"], out=st["out"])
        return {"out": out, "scale": s}
    if c["op"] == "ffn":
        return moe.expert_ffn_w8a8(st["x"], st["offsets"], st["w1"], st["s1"], st["w2"], st["s2"], y_perm=st["out"],
                                   workspace=st["workspace"], swiglu=st["swiglu"], fc1_bias=st["b1"],
                                   fc2_bias=st["b2"], fc1_layout=c["layout"])
    r = moe.balance_loss(st["logits"], st["idx"], coef=st["coef"], mask=st["mask"], seq_offsets=st["seq"])
    d = moe.balance_loss_backward(st["logits"], c["k"], r["counts"], r["tokens"], coef=st["coef"], mask=st["mask"],
                                  seq_offsets=st["seq"])
    return {"loss": r["loss"], "counts": r["counts"], "probs": r["probs"], "tokens": r["tokens"], "dlogits": d}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "product":
        return _plain_product(state)
    return _plain_ffn(state) if op == "ffn" else _plain_balance(state)


# ------------------------------------------------------- the definition, in 64 bits

def _exact_linear(x, w, ws, bias):
    """One expert: round x's rows to 8 bits with their scale, multiply, scale, add."""
    x = x.double()
    top = x.abs().max(dim=1).values
    s = (top.float() / 127).double()          # the scale is a float32 by definition
    q = torch.where(top[:, None] > 0, torch.round(x * 127 / top[:, None]), torch.zeros_like(x))
    y = (q @ w.double().T) * (s[:, None] * ws.double()[None, :])
    return (y if bias is None else y + bias.double()[None, :]), top / 127


def _exact_balance(st):
    lg, idx, coef = st["logits"].double(), st["idx"].long().cpu().numpy(), st["coef"]
    T, E = lg.shape
    k = idx.shape[1]
    p = torch.softmax(lg, dim=1)
    valid = np.ones(T, bool) if st["mask"] is None else st["mask"].cpu().numpy()
    seq = np.array([0, T]) if st["seq"] is None else st["seq"].cpu().numpy()
    S = len(seq) - 1
    loss, grad = 0.0, torch.zeros_like(lg)
    counts, tokens = np.zeros((S, E), np.int32), np.zeros((S,), np.int32)
    probs = torch.zeros((S, E), dtype=torch.float64, device=lg.device)
    for s in range(S):
        at = np.arange(seq[s], seq[s + 1])
        at = at[valid[at]]
        tokens[s] = n = len(at)
        if n == 0:
            continue
        counts[s] = np.bincount(idx[at].ravel(), minlength=E)
        f = torch.from_numpy(counts[s] / (n * k)).to(lg.device)
        f0 = f - 1.0 / E                      # sum_j p_j = 1: equal shares give a gradient of zero
        ps = p[torch.from_numpy(at).to(lg.device)]
        probs[s] = ps.mean(0)
        loss += coef / S * E * float((f * probs[s]).sum())
        grad[torch.from_numpy(at).to(lg.device)] = coef * E / (S * n) * ps * (f0[None, :] - ps @ f0[:, None])
    def dev(a):
        return torch.from_numpy(a).to(lg.device)

    return {"loss": torch.tensor([loss], dtype=torch.float64, device=lg.device), "counts": dev(counts), "probs": probs,
            "tokens": dev(tokens), "dlogits": grad}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(st)
    x = st["x"]
    off = [0, x.shape[0]] if st["offsets"] is None else st["offsets"].tolist()
    y = torch.zeros(st["out"].shape, dtype=torch.float64, device=x.device)
    scale = torch.zeros((x.shape[0],), dtype=torch.float64, device=x.device)
    dense = st["offsets"] is None
    for e, (a, b) in enumerate(zip(off[:-1], off[1:])):
        if a == b:
            continue
        if case["op"] == "product":
            w, ws, bias = st["w"], st["ws"], st["bias"]
            if not dense:
                w, ws, bias = w[e], ws[e], (None if bias is None else bias[e])
            y[a:b], scale[a:b] = _exact_linear(x[a:b], w, ws, bias)
            continue
        h, _ = _exact_linear(x[a:b], st["w1"][e], st["s1"][e], None if st["b1"] is None else st["b1"][e])
        n = case["I"]
        g, u = (h[:, :n], h[:, n:]) if case["layout"] == "chunked" else (h[:, 0::2], h[:, 1::2])
        alpha, beta, limit = st["swiglu"]
        g = torch.minimum(g, torch.full_like(g, limit))
        u = torch.maximum(torch.minimum(u, torch.full_like(u, limit)), torch.full_like(u, -limit))
        y[a:b], _ = _exact_linear(g * torch.sigmoid(alpha * g) * (u + beta), st["w2"][e], st["s2"][e],
                                  None if st["b2"] is None else st["b2"][e])
    return {"out": y, "scale": scale} if case["op"] == "product" else y
