"""Inputs and error bounds of the int8 x int8 tests, derived from the formulas.

Unit roundoffs: U32 = 2^-24 (float32), UB = 2^-8 (bf16), each relative to the value.

Product: the sum is exact; it is rounded to float32 (U32), the two scales are multiplied
(U32) and the bias added by one fused operation (U32 of the result), then the result is
rounded to the output type.  To first order |d| <= 2 U32 |S sa sw| + (U32 + U_out) |y|; a
factor 1.01 covers the second-order terms.

FFN: the gate and up values carry the product's error (no output rounding).  act =
g sigmoid(alpha g) (u + beta): |d act / d g| <= 1.1 |u + beta| (the derivative of silu is at
most 1.1, scaling alpha does not change it), |d act / d u| = |g sigmoid(alpha g)|; the
exponential's argument alpha g, its product with log2 e and log2 e itself round (|alpha g| U32
each at most, absolute in the exponent), the exponential and the quotient are within 2 ulp and
the two sums and two products add half an ulp each: (12 + 3 |alpha g|) U32 of |act| in all (an
ulp is at most 2 U32), 16 U32 taken for the first.  The int8 activation of an element can
therefore differ by one step where its quotient v = 127 a / amax lies within
delta = 127 (err_i + |a_i| / amax max err) / amax of a half, and the row's scale by
max err / amax of itself."""
import numpy as np
import torch

from oracle import moe_oracle as O

U32, UB = 2.0 ** -24, 2.0 ** -8
UOUT = {"bf16": UB, "f32": U32}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def rounded(a, dt):
    """float array -> (torch tensor of type dt, its exact float64 values)."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(TORCH[dt])
    return t, t.float().numpy().astype(np.float64)


def weights(rng, *shape):
    q = np.clip(np.rint(rng.standard_normal(shape) * 127 / 4), -127, 127).astype(np.int8)
    s = (rng.uniform(0.75, 1.25, shape[:-1]) * (4 / 127) / np.sqrt(shape[-1])).astype(np.float32)
    return q, s


def product_bound(a_q, a_s, w_q, w_s, y, dt, bias=None):
    raw = np.abs(O.matmul_q8(a_q, a_s, w_q, w_s))
    return 1.01 * (2 * U32 * raw + (U32 + UOUT[dt]) * np.abs(y)) + 1e-30


def ffn_with_bound(x, q1, s1, q2, s2, layout, act, b1=None, b2=None):
    """(y, bound) of one expert in float64 and the bound above on a kernel's bf16 result."""
    alpha, beta, limit = act
    q, s = O.quantize_rows(x)
    h = O.matmul_q8(q, s, q1, s1, b1)
    eh = 1.01 * (2 * U32 * np.abs(O.matmul_q8(q, s, q1, s1)) + U32 * np.abs(h))
    g, u = (v.T for v in O.fc1_gate_up(h.T, layout))
    eg, eu = (v.T for v in O.fc1_gate_up(eh.T, layout))
    a = O.swiglu(g, u, *act)
    gc, uc = np.minimum(g, limit), np.clip(u, -limit, limit)
    sg = np.abs(O.swiglu(g, np.ones_like(u), alpha, 0.0, limit)) if beta == 0.0 else \
        np.abs(gc / (1 + np.exp(-alpha * gc)))
    ea = 1.1 * np.abs(uc + beta) * eg + sg * eu + (16 + 3 * np.abs(alpha * gc)) * U32 * np.abs(a)
    aq, as_ = O.quantize_rows(a)
    amax = np.max(np.abs(a), axis=1, keepdims=True)
    safe = np.where(amax > 0, amax, 1.0)
    emax = np.max(ea, axis=1, keepdims=True)
    v = 127.0 * a / safe
    delta = 127.0 * (ea + np.abs(a) / safe * emax) / safe
    near = (np.abs(np.abs(v - np.trunc(v)) - 0.5) <= delta).astype(np.float64)
    y = O.matmul_q8(aq, as_, q2, s2, b2)
    flips = (near @ np.abs(q2.astype(np.float64)).T) * as_.astype(np.float64)[:, None] * s2[None, :]
    raw = np.abs(O.matmul_q8(aq, as_, q2, s2))
    # the scale: its rounding (U32) and the maximum's error; a relative 1.01 on all of it
    scale = raw * (emax / safe + U32)
    return y, 1.01 * (flips + scale) + product_bound(aq, as_, q2, s2, y, "bf16")


def check(got, ref, bound, what):
    d = np.abs(np.asarray(got, dtype=np.float64) - ref)
    bad = ~(d <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(d), np.inf, d - bound)), d.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {d.size} beyond the bound; worst at {i}: "
                             f"got {np.asarray(got)[i]!r} ref {ref[i]!r} bound {bound[i]:.3e}")


def split(rows, E, rng, skew=1.0, used=None):
    """Sizes of E experts' row blocks, some of them empty, summing to rows."""
    p = np.exp(skew * rng.standard_normal(E))
    if used is not None:
        p[rng.permutation(E)[used:]] = 0.0
    return rng.multinomial(rows, p / p.sum())
