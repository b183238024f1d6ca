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


# ---------------------------------------------------------------- 8-bit cache
def e4m3(x):
    """Nearest e4m3 value of float64 x with |x| <= 448, ties to even."""
    e = torch.frexp(x)[1] - 1  # exponent of the leading bit
    step = torch.ldexp(torch.ones_like(x), e.clamp_min(-6) - 3)
    return torch.round(x / step) * step


def block_scale(amax):
    """The smallest power of two s >= 2^-120 with amax <= 448 s."""
    s = 2.0 ** -120
    while 448 * s < amax:
        s *= 2
    return s


class Cache:
    """One sequence and KV head: values of the positions in use, and the scale of each block."""

    def __init__(self, block):
        self.block, self.x, self.scale = block, None, {}

    def append(self, pos, rows):
        """rows [n, dh] at pos..; positions behind pos + n are dropped."""
        n, dh = rows.shape
        old = torch.zeros(0, dh, dtype=torch.float64) if self.x is None else self.x[:pos]
        assert old.shape[0] == pos
        self.x = torch.cat([old, rows.double()])
        for tb in range(pos // self.block, (pos + n - 1) // self.block + 1 if n else 0):
            a, z = tb * self.block, min((tb + 1) * self.block, pos + n)
            lo = max(a, pos)
            new = self.x[lo:z]
            fine = new[torch.isfinite(new)].abs()
            s = block_scale(float(fine.max()) if fine.numel() else 0.0)
            if lo > a:
                s = max(s, self.scale[tb])
            self.scale[tb] = s
            y = torch.where(torch.isfinite(self.x[a:z]), self.x[a:z], 0.0)
            self.x[a:z] = torch.where(torch.isfinite(self.x[a:z]), e4m3(y / s) * s, math.nan)

    def scales(self):
        n = self.x.shape[0]
        return torch.tensor([self.scale[j // self.block] for j in range(n)], dtype=torch.float64)


def decode(q, k, v, vs, p, window, sinks, scale, bf16):
    """Query rows q [r, dh] at position p over k, v [L, dh] (float64; vs [L]: scale of V's block): out [r, dh],
    the weights [r, L] and the bound of out's error.

    Probabilities are rounded to half, 2^-11 of themselves, or 2^-25 of the largest probability times V scale
    where that is more (float32 rows: 2^-22 of themselves); scores are float32 sums of dh exact products."""
    L, dh = k.shape
    j = torch.arange(L)
    m = j <= p
    if window:
        m = m & ((j > p - window) | (j < sinks))
    if not m.any():
        return torch.zeros_like(q), torch.zeros(q.shape[0], L, dtype=torch.float64), torch.zeros_like(q)
    k, v, vs = k[m], v[m], vs[m]
    s = q @ k.T * scale
    w = torch.softmax(s, -1)
    out = w @ v
    ds = (dh + 8) * 2.0 ** -24 * (q.abs() @ k.abs().T).max() * scale + 2.0 ** -20
    top = (w * vs).max(-1, keepdim=True)[0]
    e = (2 * ds + (2.0 ** -11 if bf16 else 2.0 ** -22)) * (w @ v.abs()) + 2.0 ** -25 * top * (v / vs[:, None]).abs().sum(0)
    e = e + (BF16 if bf16 else 2.0 ** -23) * (out.abs() + e)
    full = torch.zeros(q.shape[0], L, dtype=torch.float64)
    full[:, m] = w
    return out, full, e


def keep_positions(weights, n, keep, first, recent):
    """The kept positions of one sequence and head, ascending; weights: n floats."""
    if n <= keep:
        return list(range(n))
    mid = sorted(range(first, n - recent), key=lambda j: (0, 0, j) if math.isnan(weights[j]) else (1, -weights[j], j))
    return list(range(first)) + sorted(mid[:keep - first - recent]) + list(range(n - recent, n))
