"""Float64 definitions of the bounded-memory attention operators and the error bounds of their tests
(plain torch on the CPU; shares nothing with the CUDA path).

A rounding to bf16 is off by at most half a step, 2^-8 of the value.  SLACK covers what float32 adds on
top: scores of up to 2^7 accumulated over d_head <= 128 products (relative 2^-17 of the sum of their
magnitudes, which the tests keep below 2^4), 2^x to 2^-22, and float32 sums over the keys.
"""
import math

import torch

BF16 = 2.0 ** -8
SLACK = 2.0 ** -11


def sees(S, window, sinks):
    t, j = torch.arange(S)[:, None], torch.arange(S)[None]
    m = j <= t
    return m & ((j > t - window) | (j < sinks)) if window else m


def window_forward(q, k, v, window, sinks, scale=None):
    """One sequence: q [S, Hq, dh], k, v [S, Hkv, dh] float64 -> out, P [Hq, S, S], lse (log2 units) [Hq, S]."""
    S, Hq, dh = q.shape
    G = Hq // k.shape[1]
    scale = 1 / math.sqrt(dh) if scale is None else scale
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("thd,jhd->htj", q, kk) * scale
    s = s.masked_fill(~sees(S, window, sinks), -math.inf)
    P = torch.softmax(s, -1)
    return torch.einsum("htj,jhd->thd", P, vv), P, torch.logsumexp(s, -1) / math.log(2)


def window_backward(q, k, v, do, window, sinks, scale=None):
    """Gradients of sum(do * out) by the formula: dq, dk, dv."""
    S, Hq, dh = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = 1 / math.sqrt(dh) if scale is None else scale
    out, P, _ = window_forward(q, k, v, window, sinks, scale)
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    dP = torch.einsum("thd,jhd->htj", do, vv)
    dS = P * (dP - (do * out).sum(-1).T[..., None]) * scale
    fold = lambda x: x.view(S, Hkv, G, dh).sum(2)  # noqa: E731
    return (torch.einsum("htj,jhd->thd", dS, kk), fold(torch.einsum("htj,thd->jhd", dS, q)),
            fold(torch.einsum("htj,thd->jhd", P, do)))


def window_bounds(q, k, v, do, window, sinks, scale=None):
    """Elementwise error bounds of out, dq, dk, dv.  P enters P V and P^T dO rounded to bf16, dS = P (dP - D)
    enters dS K and dS^T Q rounded to bf16, D is a float32 sum over the bf16 output, and every result is
    rounded to bf16 once."""
    S, Hq, dh = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = 1 / math.sqrt(dh) if scale is None else scale
    out, P, _ = window_forward(q, k, v, window, sinks, scale)
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    e_out = (BF16 + SLACK) * (torch.einsum("htj,jhd->thd", P, vv.abs()) + out.abs())
    if do is None:
        return e_out
    e_D = (do.abs() * e_out).sum(-1).T[..., None] + SLACK * (do * out).abs().sum(-1).T[..., None]
    dP = torch.einsum("thd,jhd->htj", do, vv)
    mag = torch.einsum("thd,jhd->htj", do.abs(), vv.abs())
    dS = P * (dP - (do * out).sum(-1).T[..., None])
    e_dS = scale * (P * (e_D + SLACK * mag) + (BF16 + SLACK) * (dS.abs() + P * e_D))
    fold = lambda x: x.view(S, Hkv, G, dh).sum(2)  # noqa: E731
    dq, dk, dv = window_backward(q, k, v, do, window, sinks, scale)
    tiny = 2.0 ** -126
    return (e_out, torch.einsum("htj,jhd->thd", e_dS, kk.abs()) + (BF16 + SLACK) * dq.abs() + tiny,
            fold(torch.einsum("htj,thd->jhd", e_dS, q.abs())) + (BF16 + SLACK) * dk.abs() + tiny,
            fold((BF16 + SLACK) * torch.einsum("htj,thd->jhd", P, do.abs())) + (BF16 + SLACK) * dv.abs() + tiny)
