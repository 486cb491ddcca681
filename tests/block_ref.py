"""Plain 64-bit references of the feed-forward block's operators, on the CPU
in torch float64, and the bounds that the kernels' arithmetic obeys.

U32 and UBF16 are half a step of fp32 and bf16 relative to the value; an E4M3
code is off by at most 2^-4 of its value, or half the subnormal step, 2^-10,
times its scale.
"""
import math

import numpy as np
import torch

F64 = torch.float64
U32, UBF16, UE4M3 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4
E4M3_MAX, AMAX_FLOOR = 448.0, 448.0 * 2.0 ** -126
SILU, GELU = 0, 1


def decode(q):
    """Values of E4M3 codes (uint8)."""
    return q.cpu().view(torch.float8_e4m3fn).to(F64)


def rows64(q, s):
    """Codes [M, K] in 1x128 groups with scales [K/128, M]."""
    return decode(q) * s.cpu().to(F64).repeat_interleave(128, 0).t()[: q.shape[0], : q.shape[1]]


def cols64(q, s):
    """Transposed codes [C, P] in 128x1 groups, scales [P/128, C] -> [P, C]."""
    return decode(q).t() * s.cpu().to(F64).repeat_interleave(128, 0)


def blocks64(q, s):
    return decode(q) * s.cpu().to(F64).repeat_interleave(128, 0).repeat_interleave(128, 1)


def act(g, kind):
    if kind == SILU:
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def act_grad(g, kind):
    if kind == SILU:
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)


def gated(x, w, kind):
    """(H, G, U, sum |x||w| of G and of U) from x [M, K] and stacked w [2N, K]."""
    gu, size = x @ w.t(), x.abs() @ w.abs().t()
    n = w.shape[0] // 2
    return act(gu[:, :n], kind) * gu[:, n:], gu[:, :n], gu[:, n:], size[:, :n], size[:, n:]


def gated_backward(dh, g, u, kind):
    """dG, dU, H."""
    return dh * u * act_grad(g, kind), dh * act(g, kind), act(g, kind) * u


def gate_rows_of(gate, rows, M):
    return gate.repeat_interleave(rows, 0)[:M]


def norm(x, y=None, w_post=None, gate=None, alpha=1.0, w_pre=None, eps=1e-6):
    """x', h, r_y, r_x (gate already one row per row)."""
    ry = rx = h = None
    if y is not None:
        n = y
        if w_post is not None:
            ry = (y.square().mean(1) + eps).rsqrt()
            n = y * ry[:, None] * w_post
        x = alpha * x + (n if gate is None else gate * n)
    if w_pre is not None:
        rx = (x.square().mean(1) + eps).rsqrt()
        h = x * rx[:, None] * w_pre
    return x, h, ry, rx


def norm_backward(dxo, dh, xo, rx, w_pre, y, ry, w_post, gate, gate_rows, alpha):
    """dx, dy, dw_pre, dw_post, dgate."""
    M, D = xo.shape
    t = torch.zeros(M, D, dtype=F64) if dxo is None else dxo
    dw_pre = dw_post = dgate = dy = None
    if dh is not None:
        xh = xo * rx[:, None]
        v = dh * w_pre
        dw_pre = (dh * xh).sum(0)
        t = t + rx[:, None] * (v - xh * (v * xh).mean(1, keepdim=True))
    if y is None:
        return t, None, dw_pre, None, None
    yh = y * ry[:, None] if w_post is not None else y
    n = yh * w_post if w_post is not None else y
    dn = t
    if gate is not None:
        dgate = torch.zeros_like(gate).index_add_(0, torch.arange(M) // gate_rows, t * n)
        dn = t * gate_rows_of(gate, gate_rows, M)
    dy = dn
    if w_post is not None:
        dw_post = (dn * yh).sum(0)
        z = dn * w_post
        dy = ry[:, None] * (z - yh * (z * yh).mean(1, keepdim=True))
    return alpha * t, dy, dw_pre, dw_post, dgate


def quant_rows32(x):
    """The quantisers' arithmetic on fp32 values in 1x128 groups: codes, scales [C/128, M]."""
    x = x.cpu()
    M, C = x.shape
    g = x.view(M, C // 128, 128)
    amax = g.abs().amax(2).clamp_min(AMAX_FLOOR)
    q = (g * (torch.tensor(E4M3_MAX) / amax)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn).view(torch.uint8).view(M, C), (amax / E4M3_MAX).t().contiguous()


def check_groups(q, s, x, err, pow2, tag):
    """Codes q [R, C] and scales s [R, C/128] in 1x128 groups stand for x to
    within err (elementwise, of the value before quantisation) and the
    quantisation itself."""
    q, s, x = decode(q), s.cpu().to(F64), x
    R, C = x.shape
    sg = s.repeat_interleave(128, 1)
    amax = x.abs().view(R, C // 128, 128).amax(2).clamp_min(AMAX_FLOOR)
    slack = err.view(R, C // 128, 128).amax(2)
    if pow2:
        m, _ = torch.frexp(s)
        assert bool((m == 0.5).all()), (tag, "scales are powers of two")
        assert bool((amax - slack <= 448 * s * (1 + 4 * U32)).all()), (tag, "scale too small")
        assert bool(((amax + slack) * (1 + 4 * U32) >= 224 * s).all() | (s <= 2.0 ** -125).all()), (tag, "too large")
    else:
        # the amax and one division
        assert bool(((s - amax / 448).abs() <= slack / 448 + 4 * U32 * amax / 448).all()), (tag, "scales")
    bound = err + UE4M3 * (x.abs() + err) * (1 + 8 * U32) + 2.0 ** -10 * sg + 8 * U32 * x.abs()
    off = (q * sg - x).abs()
    worst = float((off / bound.clamp_min(1e-300)).max())
    assert worst <= 1.0, (tag, "codes", worst)


def bits(t):
    t = t.detach().cpu()
    return t.view(torch.int16).numpy() if t.dtype == torch.bfloat16 else t.numpy().view(np.uint8)
