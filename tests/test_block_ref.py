"""The 64-bit references of the feed-forward block against central
differences of their forward forms (CPU)."""
import pytest
import torch

import block_ref as ref
from block_ref import F64


def numeric(f, x, h=1e-6):
    """Central differences of the scalar f at x."""
    g = torch.zeros_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + h
        up = float(f())
        flat[i] = keep - h
        out[i] = (up - float(f())) / (2 * h)
        flat[i] = keep
    return g


# differences of step h are off by f'''h^2/6 ~ 1e-11 and by rounding 2^-53 |f| / h ~ 1e-8 (|f| < 100)
TOL = 1e-6


@pytest.mark.parametrize("act", [ref.SILU, ref.GELU])
def test_gated_gradients(act):
    gen = torch.Generator().manual_seed(3)
    g, u, dh = (torch.randn(3, 5, generator=gen, dtype=F64) * 2 for _ in range(3))
    f = lambda: (ref.act(g, act) * u * dh).sum()  # noqa: E731
    dg, du, h = ref.gated_backward(dh, g, u, act)
    assert float((numeric(f, g) - dg).abs().max()) < TOL
    assert float((numeric(f, u) - du).abs().max()) < TOL
    assert torch.equal(h, ref.act(g, act) * u)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_norm_gradients(post, gated):
    gen = torch.Generator().manual_seed(4)
    M, D, rows, alpha = 5, 6, 2, 0.7
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=F64)  # noqa: E731
    x, y, dxo, dh = rnd(M, D), rnd(M, D), rnd(M, D), rnd(M, D)
    w_pre, w_post, gate = rnd(D), rnd(D) if post else None, rnd(3, D) if gated else None

    def f():
        xo, h, _, _ = ref.norm(x, y, w_post, ref.gate_rows_of(gate, rows, M) if gated else None, alpha, w_pre)
        return (xo * dxo).sum() + (h * dh).sum()
    xo, _, ry, rx = ref.norm(x, y, w_post, ref.gate_rows_of(gate, rows, M) if gated else None, alpha, w_pre)
    dx, dy, dw_pre, dw_post, dgate = ref.norm_backward(dxo, dh, xo, rx, w_pre, y, ry, w_post, gate, rows, alpha)
    for value, got in ((x, dx), (y, dy), (w_pre, dw_pre), (w_post, dw_post), (gate, dgate)):
        if value is not None:
            assert float((numeric(f, value) - got).abs().max()) < TOL
