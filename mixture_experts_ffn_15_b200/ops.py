"""Torch-facing wrappers of the C ABI.

PyTorch provides device memory and streams only: every step of the layer runs in
the CUDA kernels of libmoe_b200.so.  These functions check dtypes, devices, shapes
and contiguity, allocate outputs and workspaces with torch when the caller does
not pass them, and raise MoEError on any non-OK status.
"""
import contextlib
import ctypes

import torch

from . import _abi
from ._abi import STANDARD_SWIGLU, MoeSwiglu, check

_DT = {torch.bfloat16: _abi.MOE_BF16, torch.float32: _abi.MOE_F32}


def _lib():
    return _abi.load()


def _dtcode(t):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}: bfloat16 or float32") from None


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype=None, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _swiglu(alpha, beta, limit):
    return MoeSwiglu(alpha, beta, limit)


_LAYOUT = {"interleaved": 0, "chunked": 1}


def _layout(fc1_layout):
    if fc1_layout not in _LAYOUT:
        raise ValueError(f"fc1_layout must be 'interleaved' or 'chunked', got {fc1_layout!r}")
    return _LAYOUT[fc1_layout]


def workspace_size(T, H, E, k, I, dtype):
    """Bytes of workspace moe_forward needs (0 for sizes it rejects)."""
    return _lib().moe_workspace_size(T, H, E, k, I, _DT[dtype])


def alloc_workspace(nbytes, device):
    """Device workspace, zero-filled (moe_forward wants zeros before its first call)."""
    return torch.zeros(int(nbytes), dtype=torch.uint8, device=device)


def _biases(fc1_bias, fc2_bias, dt, E, I, H):
    if fc1_bias is not None:
        _need(fc1_bias, "fc1_bias", dt, (E, 2 * I))
    if fc2_bias is not None:
        _need(fc2_bias, "fc2_bias", dt, (E, H))


def forward(hidden, router_w, fc1, fc2, k, normalize=True, router_bias=None, out=None,
            workspace=None, stream=None, swiglu=(1.0, 0.0, float("inf")), fc1_bias=None,
            fc2_bias=None, fc1_layout="interleaved", norm_weight=None, norm_eps=1e-6):
    """The fused MoE layer: out[T, H] = sum_j w[t, j] * FFN_{idx[t, j]}(hidden[t]).

    swiglu = (alpha, beta, limit) of the op; fc1_layout "interleaved" (rows 2i, 2i+1 =
    gate_i, up_i) or "chunked" (rows i, I+i), read in place either way; fc1_bias
    [E, 2I] (fc1's layout) and fc2_bias [E, H] are the optional expert biases.  With
    norm_weight [H], hidden is the residual activation and the layer runs on its
    pre-FFN RMSNorm (computed inside the call, see rmsnorm)."""
    _need(hidden, "hidden")
    dt = hidden.dtype
    T, H = hidden.shape
    E = router_w.shape[0]
    I = fc2.shape[2]
    _need(router_w, "router_w", dt, (E, H))
    _need(fc1, "fc1", dt, (E, 2 * I, H))
    _need(fc2, "fc2", dt, (E, H, I))
    if router_bias is not None:
        _need(router_bias, "router_bias", torch.float32, (E,))
    _biases(fc1_bias, fc2_bias, dt, E, I, H)
    if norm_weight is not None:
        _need(norm_weight, "norm_weight", dt, (H,))
    if out is None:
        out = torch.empty_like(hidden)
    _need(out, "out", dt, (T, H))
    need = workspace_size(T, H, E, k, I, dt)
    if workspace is None:
        # invalid sizes give 0 bytes; the C call then reports them
        workspace = alloc_workspace(max(need, 256), hidden.device)
    _need(workspace, "workspace", torch.uint8)
    st = _lib().moe_forward(_ptr(hidden), _ptr(norm_weight), float(norm_eps), _ptr(router_w),
                            _ptr(router_bias), _ptr(fc1), _ptr(fc2),
                            _ptr(fc1_bias), _ptr(fc2_bias), T, H, E, k, I, int(bool(normalize)),
                            _swiglu(*swiglu), _layout(fc1_layout), _dtcode(hidden), _ptr(out),
                            _ptr(workspace),
                            workspace.numel(), _stream(stream))
    check(st, "moe_forward")
    return out


def _q8(q, scale, name, rows_shape):
    _need(q, name, torch.int8, rows_shape)
    _need(scale, name + "_scale", torch.float32, rows_shape[:2])


def forward_q8(hidden, router_w, fc1_q, fc1_scale, fc2_q, fc2_scale, k, normalize=True,
               router_bias=None, out=None, workspace=None, stream=None,
               swiglu=(1.0, 0.0, float("inf")), fc1_bias=None, fc2_bias=None,
               fc1_layout="interleaved", norm_weight=None, norm_eps=1e-6):
    """The layer with weight-only int8 experts: weight = q * scale of its row (fc1_q
    [E, 2I, H] int8 with fc1_scale [E, 2I] float32, fc2_q [E, H, I] with fc2_scale
    [E, H]); hidden and the rest bf16, as in forward.  Decode-sized batches only."""
    _need(hidden, "hidden", torch.bfloat16)
    T, H = hidden.shape
    E = router_w.shape[0]
    I = fc2_q.shape[2]
    _need(router_w, "router_w", torch.bfloat16, (E, H))
    _q8(fc1_q, fc1_scale, "fc1", (E, 2 * I, H))
    _q8(fc2_q, fc2_scale, "fc2", (E, H, I))
    if router_bias is not None:
        _need(router_bias, "router_bias", torch.float32, (E,))
    _biases(fc1_bias, fc2_bias, torch.bfloat16, E, I, H)
    if norm_weight is not None:
        _need(norm_weight, "norm_weight", torch.bfloat16, (H,))
    if out is None:
        out = torch.empty_like(hidden)
    _need(out, "out", torch.bfloat16, (T, H))
    need = workspace_size(T, H, E, k, I, torch.bfloat16)
    if workspace is None:
        workspace = alloc_workspace(max(need, 256), hidden.device)
    _need(workspace, "workspace", torch.uint8)
    st = _lib().moe_forward_q8(_ptr(hidden), _ptr(norm_weight), float(norm_eps), _ptr(router_w),
                               _ptr(router_bias), _ptr(fc1_q), _ptr(fc1_scale), _ptr(fc2_q),
                               _ptr(fc2_scale), _ptr(fc1_bias), _ptr(fc2_bias), T, H, E, k, I,
                               int(bool(normalize)), _swiglu(*swiglu), _layout(fc1_layout),
                               _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    check(st, "moe_forward_q8")
    return out


def expert_ffn_q8(x_perm, offsets, fc1_q, fc1_scale, fc2_q, fc2_scale, y_perm=None, stream=None,
                  swiglu=(1.0, 0.0, float("inf")), fc1_bias=None, fc2_bias=None,
                  fc1_layout="interleaved"):
    """expert_ffn with weight-only int8 experts (see forward_q8)."""
    _need(x_perm, "x_perm", torch.bfloat16)
    rows, H = x_perm.shape
    E, two_i, _ = fc1_q.shape
    I = two_i // 2
    _need(offsets, "offsets", torch.int32, (E + 1,))
    _q8(fc1_q, fc1_scale, "fc1", (E, 2 * I, H))
    _q8(fc2_q, fc2_scale, "fc2", (E, H, I))
    _biases(fc1_bias, fc2_bias, torch.bfloat16, E, I, H)
    if y_perm is None:
        y_perm = torch.zeros_like(x_perm)
    ws = alloc_workspace(_lib().moe_expert_ffn_workspace_size(rows, I, _DT[torch.bfloat16]),
                         x_perm.device)
    st = _lib().moe_expert_ffn_q8(_ptr(x_perm), _ptr(offsets), _ptr(fc1_q), _ptr(fc1_scale),
                                  _ptr(fc2_q), _ptr(fc2_scale), _ptr(fc1_bias), _ptr(fc2_bias), rows,
                                  H, E, I, _swiglu(*swiglu), _layout(fc1_layout), _ptr(y_perm),
                                  _ptr(ws), ws.numel(), _stream(stream))
    check(st, "moe_expert_ffn_q8")
    return y_perm


def _same_device(t, *others):
    dev = t.device
    for o in others:
        if o is not None and o.device != dev:
            raise ValueError(f"every tensor must be on {dev}, got one on {o.device}")


def _addr(t):
    return None if t is None else t.data_ptr()


_HERE = contextlib.nullcontext()
# The current stream's handle of a device: 0.1 us, a Stream object 3 us.  (A torch build without
# CUDA lacks the function; the package imports there, for the C library and the checks.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda i: torch.cuda.current_stream(i).cuda_stream)


def _on(t, stream):
    """(stream handle, context) of a call: the caller's stream, or the current one of t's
    device.  What is allocated inside the context belongs to that stream; the context is
    empty where the stream is the current one already."""
    if stream is None:
        i = t.device.index
        return _raw_stream(i), (_HERE if i == torch.cuda.current_device() else torch.cuda.device(i))
    if stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {t.device}")
    return stream.cuda_stream, torch.cuda.stream(stream)


def quantize_rows(x, q=None, scale=None, stream=None):
    """x [rows, K] (bf16 or float32) -> (q [rows, K] int8, scale [rows] float32): per row
    scale = max|x| / 127 and q = 127 x / max|x| to the nearest whole number, ties to even
    (exact).  A zero row gives scale 0 and q 0; one with an infinity or a NaN scale NaN
    and q 0."""
    _need(x, "x")
    rows, K = x.shape
    s, here = _on(x, stream)
    with here:
        if q is None:
            q = torch.empty_like(x, dtype=torch.int8)
        else:
            _same_device(x, _need(q, "q", torch.int8, (rows, K)))
        if scale is None:
            scale = x.new_empty(rows, dtype=torch.float32)
        else:
            _same_device(x, _need(scale, "scale", torch.float32, (rows,)))
        check(_lib().moe_quantize_rows(x.data_ptr(), rows, K, _dtcode(x), q.data_ptr(),
                                       scale.data_ptr(), s), "moe_quantize_rows")
    return q, scale


def matmul_q8(a_q, a_scale, w_q, w_scale, offsets=None, bias=None, out=None,
              out_dtype=torch.bfloat16, err_word=None, stream=None):
    """out[r, n] = (sum_k a_q[r, k] w_q[e, n, k]) a_scale[r] w_scale[e, n] + bias[e, n]:
    int8 rows (quantize_rows) times int8 weights, the sum exact.  Dense (w_q [N, K],
    w_scale and bias [N]) or, with offsets [E+1], grouped: rows offsets[e] ..
    offsets[e+1]-1 meet w_q[e] of w_q [E, N, K] (w_scale and bias [E, N]); rows at or
    beyond offsets[E] are not written (zeros when out is not given).  out, and bias, are
    bf16 or float32 (out_dtype, or out's own)."""
    _need(a_q, "a_q", torch.int8)
    rows, K = a_q.shape
    _need(a_scale, "a_scale", torch.float32, (rows,))
    grouped = offsets is not None
    if w_q.dim() != (3 if grouped else 2):
        raise ValueError("w_q must be [E, N, K] with offsets, [N, K] without")
    E, N = (w_q.shape[0], w_q.shape[1]) if grouped else (1, w_q.shape[0])
    lead = (E, N) if grouped else (N,)
    _need(w_q, "w_q", torch.int8, lead + (K,))
    _need(w_scale, "w_scale", torch.float32, lead)
    if grouped:
        _need(offsets, "offsets", torch.int32, (E + 1,))
    if err_word is not None:
        _need(err_word, "err_word", torch.int32)
    s, here = _on(a_q, stream)
    with here:
        if out is None:
            out = (torch.zeros if grouped else torch.empty)((rows, N), dtype=out_dtype, device=a_q.device)
        dt = _dtcode(out)
        _need(out, "out", None, (rows, N))
        if bias is not None:
            _need(bias, "bias", out.dtype, lead)
        _same_device(a_q, a_scale, w_q, w_scale, offsets, bias, out, err_word)
        check(_lib().moe_matmul_q8(_addr(a_q), _addr(a_scale), _addr(w_q), _addr(w_scale), _addr(bias),
                                   _addr(offsets), rows, K, E, N, dt, _addr(out), _addr(err_word),
                                   s), "moe_matmul_q8")
    return out


def expert_ffn_w8a8_workspace_size(rows, H, E, I):
    """Bytes of workspace expert_ffn_w8a8 needs (0 for sizes it rejects)."""
    return _lib().moe_expert_ffn_w8a8_workspace_size(rows, H, E, I)


def expert_ffn_w8a8(x_perm, offsets, fc1_q, fc1_scale, fc2_q, fc2_scale, y_perm=None,
                    workspace=None, stream=None, swiglu=(1.0, 0.0, float("inf")), fc1_bias=None,
                    fc2_bias=None, fc1_layout="interleaved"):
    """expert_ffn with int8 weights and int8 activations (quantize_rows before either
    product), for any number of rows per expert; weights and scales as in forward_q8.
    Rows at or beyond offsets[E] are not written (zeros when y_perm is not given).  The
    workspace's first word is the call's error word (get_error), zero after an empty call too."""
    _need(x_perm, "x_perm", torch.bfloat16)
    rows, H = x_perm.shape
    E, two_i, _ = fc1_q.shape
    I = two_i // 2
    _need(offsets, "offsets", torch.int32, (E + 1,))
    _q8(fc1_q, fc1_scale, "fc1", (E, 2 * I, H))
    _q8(fc2_q, fc2_scale, "fc2", (E, H, I))
    _biases(fc1_bias, fc2_bias, torch.bfloat16, E, I, H)
    s, here = _on(x_perm, stream)
    with here:
        if y_perm is None:
            y_perm = torch.zeros_like(x_perm)
        _need(y_perm, "y_perm", torch.bfloat16, (rows, H))
        if workspace is None:
            workspace = torch.empty(max(expert_ffn_w8a8_workspace_size(rows, H, E, I), 256),
                                    dtype=torch.uint8, device=x_perm.device)
        _need(workspace, "workspace", torch.uint8)
        _same_device(x_perm, offsets, fc1_q, fc1_scale, fc2_q, fc2_scale, fc1_bias, fc2_bias,
                     y_perm, workspace)
        if rows == 0:   # the C call is a no-op then
            workspace[:4].zero_()
        check(_lib().moe_expert_ffn_w8a8(_addr(x_perm), _addr(offsets), _addr(fc1_q), _addr(fc1_scale),
                                         _addr(fc2_q), _addr(fc2_scale), _addr(fc1_bias),
                                         _addr(fc2_bias), rows, H, E, I, _swiglu(*swiglu),
                                         _layout(fc1_layout), _addr(y_perm), _addr(workspace),
                                         workspace.numel(), s), "moe_expert_ffn_w8a8")
    return y_perm


def w8a8_workspace_size(T, H, E, k, I):
    """Bytes of workspace forward_w8a8 needs (0 for sizes it rejects)."""
    return _lib().moe_w8a8_workspace_size(T, H, E, k, I)


def forward_w8a8(hidden, router_w, fc1_q, fc1_scale, fc2_q, fc2_scale, k, normalize=True,
                 router_bias=None, out=None, workspace=None, stream=None,
                 swiglu=(1.0, 0.0, float("inf")), fc1_bias=None, fc2_bias=None,
                 fc1_layout="interleaved", norm_weight=None, norm_eps=1e-6):
    """The layer with int8 experts and int8 activations in the expert products (the router
    reads the bf16 input): arguments as forward_q8, any batch size.  The workspace's first
    word is the call's error word (get_error), zero after an empty call too."""
    _need(hidden, "hidden", torch.bfloat16)
    T, H = hidden.shape
    E = router_w.shape[0]
    I = fc2_q.shape[2]
    _need(router_w, "router_w", torch.bfloat16, (E, H))
    _q8(fc1_q, fc1_scale, "fc1", (E, 2 * I, H))
    _q8(fc2_q, fc2_scale, "fc2", (E, H, I))
    if router_bias is not None:
        _need(router_bias, "router_bias", torch.float32, (E,))
    _biases(fc1_bias, fc2_bias, torch.bfloat16, E, I, H)
    if norm_weight is not None:
        _need(norm_weight, "norm_weight", torch.bfloat16, (H,))
    s, here = _on(hidden, stream)
    with here:
        if out is None:
            out = torch.empty_like(hidden)
        _need(out, "out", torch.bfloat16, (T, H))
        if workspace is None:
            workspace = torch.empty(max(w8a8_workspace_size(T, H, E, k, I), 256), dtype=torch.uint8,
                                    device=hidden.device)
        _need(workspace, "workspace", torch.uint8)
        _same_device(hidden, router_w, router_bias, fc1_q, fc1_scale, fc2_q, fc2_scale, fc1_bias,
                     fc2_bias, norm_weight, out, workspace)
        if T == 0:   # the C call is a no-op then
            workspace[:4].zero_()
        check(_lib().moe_forward_w8a8(_addr(hidden), _addr(norm_weight), float(norm_eps),
                                      _addr(router_w), _addr(router_bias), _addr(fc1_q),
                                      _addr(fc1_scale), _addr(fc2_q), _addr(fc2_scale), _addr(fc1_bias),
                                      _addr(fc2_bias), T, H, E, k, I, int(bool(normalize)),
                                      _swiglu(*swiglu), _layout(fc1_layout), _addr(out),
                                      _addr(workspace), workspace.numel(), s),
              "moe_forward_w8a8")
    return out


def _balance_batch(logits, mask, seq_offsets):
    _need(logits, "logits", torch.float32)
    T, E = logits.shape
    if mask is not None:
        if mask.dtype == torch.bool:
            mask = mask.view(torch.uint8)
        _need(mask, "mask", torch.uint8, (T,))
    S = 1
    if seq_offsets is not None:
        _need(seq_offsets, "seq_offsets", torch.int32)
        if seq_offsets.dim() != 1 or seq_offsets.numel() < 2:
            raise ValueError("seq_offsets must be [S + 1] with S >= 1")
        S = seq_offsets.numel() - 1
    return T, E, S, mask


def balance_loss(logits, topk_idx, coef=1.0, mask=None, seq_offsets=None, err_word=None,
                 workspace=None, stream=None):
    """Load-balance loss of a routing (route's logits and idx) and its per-expert counts:
    with n valid tokens, f_e = counts_e / (n k) and P_e the mean softmax probability,
    coef E sum_e f_e P_e, averaged over the sequences seq_offsets [S+1] cuts the batch
    into (default: one).  mask [T] (bool or uint8): False leaves a token (padding) out.
    Returns loss [1], counts [S, E] int32, probs [S, E] (P) and tokens [S] int32 (n)."""
    T, E, S, mask = _balance_batch(logits, mask, seq_offsets)
    _need(topk_idx, "topk_idx", torch.int32)
    if topk_idx.dim() != 2 or topk_idx.shape[0] != T:
        raise ValueError(f"topk_idx must be [{T}, k], got {tuple(topk_idx.shape)}")
    if err_word is not None:
        _need(err_word, "err_word", torch.int32)
    s, here = _on(logits, stream)
    with here:
        loss, probs = logits.new_empty((1,)), logits.new_empty((S, E))
        counts = logits.new_empty((S, E), dtype=torch.int32)
        tokens = logits.new_empty((S,), dtype=torch.int32)
        if workspace is None:
            workspace = logits.new_empty((max(_lib().moe_balance_loss_workspace_size(T, E, S), 256),),
                                         dtype=torch.uint8)
        _need(workspace, "workspace", torch.uint8)
        _same_device(logits, topk_idx, mask, seq_offsets, err_word, workspace)
        check(_lib().moe_balance_loss(_addr(logits), _addr(topk_idx), _addr(mask), _addr(seq_offsets),
                                      T, E, topk_idx.shape[1], S, float(coef), _addr(loss),
                                      _addr(counts), _addr(probs), _addr(tokens), _addr(err_word),
                                      _addr(workspace), workspace.numel(), s),
              "moe_balance_loss")
    return dict(loss=loss, counts=counts, probs=probs, tokens=tokens)


def balance_loss_backward(logits, k, counts, tokens, coef=1.0, mask=None, seq_offsets=None,
                          grad_loss=None, dlogits=None, stream=None):
    """Gradient of balance_loss with respect to the logits (the counts are constants), for
    the same logits, coef, mask and seq_offsets and the counts and tokens it returned;
    grad_loss [1] float32 is the gradient arriving at the loss (default 1).  Tokens that
    take no part get zeros."""
    T, E, S, mask = _balance_batch(logits, mask, seq_offsets)
    _need(counts, "counts", torch.int32, (S, E))
    _need(tokens, "tokens", torch.int32, (S,))
    if grad_loss is not None:
        _need(grad_loss, "grad_loss", torch.float32)
        if grad_loss.numel() != 1:
            raise ValueError("grad_loss must hold one value")
    s, here = _on(logits, stream)
    with here:
        if dlogits is None:
            dlogits = torch.empty_like(logits)
        _need(dlogits, "dlogits", torch.float32, (T, E))
        _same_device(logits, counts, tokens, mask, seq_offsets, grad_loss, dlogits)
        check(_lib().moe_balance_loss_backward(_addr(logits), _addr(mask), _addr(seq_offsets),
                                               _addr(counts), _addr(tokens), T, E, int(k), S,
                                               float(coef), _addr(grad_loss), _addr(dlogits),
                                               s), "moe_balance_loss_backward")
    return dlogits


def rmsnorm(x, weight, eps=1e-6, out=None, stream=None):
    """Pre-FFN RMSNorm: (x / sqrt(mean(x^2) + eps)) * weight per row, float64 inside,
    rounded once to x's dtype."""
    _need(x, "x")
    T, H = x.shape
    _need(weight, "weight", x.dtype, (H,))
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", x.dtype, (T, H))
    check(_lib().moe_rmsnorm(_ptr(x), _ptr(weight), T, H, float(eps), _dtcode(x), _ptr(out),
                             _stream(stream)), "moe_rmsnorm")
    return out


def workspace_error_word(workspace):
    """The int32 error word at the start of a moe_forward workspace, as a tensor view."""
    return workspace[:4].view(torch.int32)


def route(hidden, router_w, k, normalize=True, router_bias=None, stream=None):
    """Router logits, top-k (descending, ties to the lower index) and routing weights."""
    _need(hidden, "hidden")
    T, H = hidden.shape
    E = router_w.shape[0]
    _need(router_w, "router_w", hidden.dtype, (E, H))
    if router_bias is not None:
        _need(router_bias, "router_bias", torch.float32, (E,))
    dev = hidden.device
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    logits = torch.empty((T, E), dtype=torch.float32, device=dev)
    near = torch.empty((T,), dtype=torch.int32, device=dev)
    st = _lib().moe_route(_ptr(hidden), _ptr(router_w), _ptr(router_bias), T, H, E, k,
                          int(bool(normalize)), _dtcode(hidden), _ptr(idx), _ptr(w), _ptr(logits),
                          _ptr(near), _stream(stream))
    check(st, "moe_route")
    return dict(idx=idx, w=w, logits=logits, near_tie=near)


def permute(topk_idx, E, hidden=None, err_word=None, stream=None):
    """Bincount, offsets, stable permutation and (with hidden) the gathered rows."""
    _need(topk_idx, "topk_idx", torch.int32)
    T, k = topk_idx.shape
    dev = topk_idx.device
    H = hidden.shape[1] if hidden is not None else 8
    dt = _dtcode(hidden) if hidden is not None else _abi.MOE_BF16
    counts = torch.empty((E,), dtype=torch.int32, device=dev)
    offsets = torch.empty((E + 1,), dtype=torch.int32, device=dev)
    perm_src = torch.full((T * k,), -1, dtype=torch.int32, device=dev)
    perm_dst = torch.empty((T * k,), dtype=torch.int32, device=dev)
    x_perm = None
    if hidden is not None:
        _need(hidden, "hidden")
        x_perm = torch.empty((T * k, H), dtype=hidden.dtype, device=dev)
    if err_word is None:
        err_word = torch.zeros((1,), dtype=torch.int32, device=dev)
    ws = alloc_workspace(_lib().moe_permute_workspace_size(T, E), dev)
    st = _lib().moe_permute(_ptr(hidden), _ptr(topk_idx), T, H, E, k, dt, _ptr(counts),
                            _ptr(offsets), _ptr(perm_src), _ptr(perm_dst), _ptr(x_perm),
                            _ptr(err_word), _ptr(ws), ws.numel(), _stream(stream))
    check(st, "moe_permute")
    return dict(counts=counts, offsets=offsets, perm_src=perm_src, perm_dst=perm_dst,
                x_perm=x_perm, err_word=err_word)


def expert_ffn(x_perm, offsets, fc1, fc2, y_perm=None, stream=None,
               swiglu=(1.0, 0.0, float("inf")), fc1_bias=None, fc2_bias=None,
               fc1_layout="interleaved"):
    """y_perm[r] = fc2_e act(x fc1_gate^T + b_gate, x fc1_up^T + b_up) + b2_e over each
    expert's rows (act: SwiGLU with the op's (alpha, beta, limit); fc1 and fc1_bias in
    fc1_layout, "interleaved" or "chunked")."""
    _need(x_perm, "x_perm")
    rows, H = x_perm.shape
    E, two_i, _ = fc1.shape
    I = two_i // 2
    _need(offsets, "offsets", torch.int32, (E + 1,))
    _need(fc1, "fc1", x_perm.dtype, (E, 2 * I, H))
    _need(fc2, "fc2", x_perm.dtype, (E, H, I))
    _biases(fc1_bias, fc2_bias, x_perm.dtype, E, I, H)
    if y_perm is None:
        y_perm = torch.zeros_like(x_perm)
    dt = _dtcode(x_perm)
    ws = alloc_workspace(_lib().moe_expert_ffn_workspace_size(rows, I, dt), x_perm.device)
    st = _lib().moe_expert_ffn(_ptr(x_perm), _ptr(offsets), _ptr(fc1), _ptr(fc2), _ptr(fc1_bias),
                               _ptr(fc2_bias), rows, H, E, I, _swiglu(*swiglu),
                               _layout(fc1_layout), dt, _ptr(y_perm),
                               _ptr(ws), ws.numel(), _stream(stream))
    check(st, "moe_expert_ffn")
    return y_perm


def combine(y_perm, perm_dst, topk_w, T, k, out=None, stream=None):
    """out[t] = sum_j topk_w[t, j] * y_perm[perm_dst[t*k + j]] (float32 sum, slot order)."""
    _need(y_perm, "y_perm")
    H = y_perm.shape[1]
    _need(perm_dst, "perm_dst", torch.int32)
    _need(topk_w, "topk_w", torch.float32)
    if out is None:
        out = torch.empty((T, H), dtype=y_perm.dtype, device=y_perm.device)
    st = _lib().moe_combine(_ptr(y_perm), _ptr(perm_dst), _ptr(topk_w), T, H, k, _dtcode(y_perm),
                            _ptr(out), _stream(stream))
    check(st, "moe_combine")
    return out


def convert_chunked_to_interleaved(src, dst=None, stream=None):
    """[E, 2I, H] gate-rows-then-up-rows -> interleaved (row 2j gate_j, row 2j+1 up_j)."""
    _need(src, "src")
    E, two_i, H = src.shape
    if dst is None:
        dst = torch.empty_like(src)
    _need(dst, "dst", src.dtype, src.shape)
    st = _lib().convert_chunked_to_interleaved(_ptr(src), _ptr(dst), E, two_i // 2, H,
                                               _dtcode(src), _stream(stream))
    check(st, "convert_chunked_to_interleaved")
    return dst


def get_error(err_word, stream=None):
    """(status, bits) of a device error word; synchronises the stream."""
    bits = ctypes.c_int32(0)
    st = _lib().moe_get_error(_ptr(err_word), _stream(stream), ctypes.byref(bits))
    return st, bits.value


def set_stage_events(events):
    """Record 6 cudaEvent handles around the stages of every moe_forward (None: off)."""
    lib = _lib()
    if events is None:
        check(lib.moe_set_stage_events(None, 0), "moe_set_stage_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e) for e in events])
    check(lib.moe_set_stage_events(arr, len(events)), "moe_set_stage_events")
