"""The feed-forward block around the FP8 GEMMs: gated products and their
backward pass, the norms at the seam between two blocks, gradient clipping.

As the rest of the binding, argument marshalling only; the contracts stand in
include/fp8bs.h.  Tensors have to live on the current device, and every call
is enqueued on its current stream.
"""
import collections
import ctypes

import torch

from . import (ACCUM_FP32, ACCUM_MFMA8_POW2, OUT_BF16, OUT_F32, SCALE_FP32, _check, _check_pow2_mode, _ptr, _stream,
               grouped_col_bound, lib)

ACT_SILU, ACT_GELU = 0, 1

BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def declare(L):
    """Argument types of this part of the C ABI."""
    i64, vp, i32, f32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    gated = [vp, i64, vp, i64, vp, i64, vp, i64, i32]
    kept = [vp, i64, i32]
    quant = [i32, vp, i64, vp, i64]
    for name, res, args in [
            ("fp8_gated_workspace_bytes", sz, [i64] * 3),
            ("fp8_gated_gemm", i32, [i64] * 3 + gated + [vp, i64, i32] + kept + [vp, sz, vp]),
            ("fp8_gated_gemm_quant", i32, [i64] * 3 + gated + quant + kept + [vp, sz, vp]),
            ("fp8_grouped_gated_gemm", i32,
             [i32, i64, i64, i64, vp, vp, i64, vp, i64, vp, vp, i32, vp, i64, i32] + kept + [vp]),
            ("fp8_grouped_gated_gemm_quant", i32,
             [i32, i64, i64, i64, vp, vp, i64, vp, i64, vp, vp, i32] + quant + kept + [vp]),
            ("fp8_gated_backward", i32, [i64, i64, vp, i64, vp, i64, i32, i32] + [vp, i64] * 6 + [vp]),
            ("fp8_grouped_gated_backward", i32,
             [i32, vp, i64, i64, vp, i64, vp, i64, i32, i32] + [vp, i64] * 6 + [vp]),
            ("fp8_norm_residual", i32, [i64, i64, vp, i64, vp, i64, vp, vp, i64, f32, f32, vp, i64, vp, vp, i64, i32,
                                        vp, i64, vp, i64, vp, vp, vp]),
            ("fp8_norm_backward_workspace_bytes", sz, [i64, i64]),
            ("fp8_norm_residual_backward", i32, [i64, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, vp, vp, i64,
                                                 f32, vp, i64, vp, i64, vp, vp, vp, vp, sz, vp]),
            ("fp8_grad_workspace_bytes", sz, [i64]),
            ("fp8_grad_norm", i32, [i64, vp, vp, vp, vp, vp, sz, vp]),
            ("fp8_grad_clip", i32, [i64, vp, vp, vp, f32, vp, vp, vp, vp, sz, vp])]:
        f = getattr(L, name)
        f.restype, f.argtypes = res, args


def _need(t, name, dtype, *shape):
    """Checks a tensor the kernels will address: on the current device, of the
    type, of the shape (an entry None is free; an int is a lower bound in the
    first dimension and exact in the last), its last dimension contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is {torch.cuda.current_device()}")
    size = t.shape
    if len(size) != len(shape):
        raise ValueError(f"{name} must have {len(shape)} dimensions, got {tuple(size)}")
    last = len(shape) - 1
    for i, want in enumerate(shape):
        if want is not None and (size[i] != want if i == last else size[i] < want):
            raise ValueError(f"{name} has shape {tuple(size)}, needs {shape}")
    if size[last] > 1 and t.stride(last) != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")


def _ld(t):
    """Leading dimension of a matrix; of one row, any that the library takes."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1] + -t.shape[1] % 16)


def _new(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


def gated_workspace_bytes(M, N, K):
    return int(lib().fp8_gated_workspace_bytes(M, N, K))


# ---- gated products ------------------------------------------------------------------

def _gated_operands(a, sa, b, sb, accum, rows=None, offsets=None):
    """Checks the operands; returns (M, N, K, G or None)."""
    _need(a, "a", U8, None, None)
    K = a.shape[1]
    M = a.shape[0] if rows is None else int(rows)
    if not 0 <= M <= a.shape[0]:
        raise ValueError(f"rows_bound {M} outside the {a.shape[0]} rows of a")
    _need(sa, "sa", F32, K // 128, None)
    if sa.shape[1] < M:
        raise ValueError(f"sa has {sa.shape[1]} rows' scales, needs {M}")
    if offsets is None:
        _need(b, "b", U8, None, K)
        G, R = None, b.shape[0]
        _need(sb, "sb", F32, R // 128, K // 128)
    else:
        _need(offsets, "offsets", I32, None)
        G = offsets.shape[0] - 1
        _need(b, "b", U8, G, None, K)
        R = b.shape[1]
        _need(sb, "sb", F32, G, R // 128, K // 128)
        if G < 0 or b.shape[0] != G or not b.is_contiguous() or not sb.is_contiguous() or sb.shape[1] != R // 128:
            raise ValueError("b and sb must be contiguous [G, 2N, K] / [G, 2N/128, K/128], offsets [G + 1]")
    if R % 2:
        raise ValueError("b must stack as many up rows as gate rows")
    if accum == ACCUM_MFMA8_POW2:
        flat = sb if G is None else sb.view(-1, sb.shape[2])
        _check_pow2_mode(accum, sa, M, flat, 0, _ld(flat), 1, flat.shape[0] * 128, K // 128)
    return M, R // 2, K, G


def _gated_kept(gu, save_gu, M, N, a):
    if gu is None and save_gu:
        gu = _new((a.shape[0], 2 * N), BF16, a)
    if gu is not None:
        _need(gu, "gu", BF16, M, 2 * N)
    return gu


def _gated_workspace(workspace, M, N, K, a):
    need = gated_workspace_bytes(M, N, K)
    if need == 0:
        return None, 0
    if workspace is None:
        workspace = _new((need,), U8, a)
    _need(workspace, "workspace", U8, None)
    return workspace, workspace.numel()


def fp8_gated_gemm(a, sa, b, sb, act=ACT_SILU, out_dtype=OUT_BF16, d=None, gu=None, save_gu=False, workspace=None,
                   accum=ACCUM_FP32):
    """H = act(X Wg^T) * (X Wu^T).  a [M, K] codes, sa [K/128, M]; b [2N, K]
    codes (gate rows, then up rows), sb [2N/128, K/128].  Returns (d [M, N],
    gu [M, 2N] bf16 pre-activations or None)."""
    M, N, K, _ = _gated_operands(a, sa, b, sb, accum)
    dt = F32 if out_dtype == OUT_F32 else BF16
    if d is None:
        d = _new((M, N), dt, a)
    else:
        _need(d, "d", dt, M, N)
    gu = _gated_kept(gu, save_gu, M, N, a)
    ws, ws_bytes = _gated_workspace(workspace, M, N, K, a)
    _check(lib().fp8_gated_gemm(M, N, K, _ptr(a), _ld(a), _ptr(sa), _ld(sa), _ptr(b), _ld(b), _ptr(sb), _ld(sb), act,
                                _ptr(d), _ld(d), out_dtype, _ptr(gu), _ld(gu) if gu is not None else 0, accum,
                                _ptr(ws), ws_bytes, _stream()), "fp8_gated_gemm")
    return d, gu


def _quant_out(q, s, M, N, a, rows):
    if q is None:
        q = _new((rows, N), U8, a)
    else:
        _need(q, "q", U8, M, N)
    if s is None:
        s = _new((N // 128, rows), F32, a)
    else:
        _need(s, "s", F32, N // 128, None)
        if s.shape[1] < M:
            raise ValueError(f"s has room for {s.shape[1]} rows' scales, needs {M}")
    return q, s


def fp8_gated_gemm_quant(a, sa, b, sb, act=ACT_SILU, scale_mode=SCALE_FP32, q=None, s=None, gu=None, save_gu=False,
                         workspace=None, accum=ACCUM_FP32):
    """fp8_gated_gemm with H quantised 1x128: returns (q [M, N], s [N/128, M],
    gu or None)."""
    M, N, K, _ = _gated_operands(a, sa, b, sb, accum)
    q, s = _quant_out(q, s, M, N, a, M)
    gu = _gated_kept(gu, save_gu, M, N, a)
    ws, ws_bytes = _gated_workspace(workspace, M, N, K, a)
    _check(lib().fp8_gated_gemm_quant(M, N, K, _ptr(a), _ld(a), _ptr(sa), _ld(sa), _ptr(b), _ld(b), _ptr(sb), _ld(sb),
                                      act, scale_mode, _ptr(q), _ld(q), _ptr(s), _ld(s), _ptr(gu),
                                      _ld(gu) if gu is not None else 0, accum, _ptr(ws), ws_bytes, _stream()),
           "fp8_gated_gemm_quant")
    return q, s, gu


def fp8_grouped_gated_gemm(offsets, a, sa, b, sb, act=ACT_SILU, out_dtype=OUT_BF16, rows_bound=None, d=None, gu=None,
                           save_gu=False, accum=ACCUM_FP32):
    """fp8_gated_gemm over experts: rows offsets[e]..offsets[e+1]-1 of a use
    b[e] [2N, K] and sb[e].  Rows at and after offsets[-1] are left as they
    are.  Returns (d, gu or None)."""
    M, N, K, G = _gated_operands(a, sa, b, sb, accum, rows_bound, offsets)
    dt = F32 if out_dtype == OUT_F32 else BF16
    if d is None:
        d = _new((M, N), dt, a)
    else:
        _need(d, "d", dt, M, N)
    gu = _gated_kept(gu, save_gu, M, N, a)
    _check(lib().fp8_grouped_gated_gemm(G, M, N, K, _ptr(offsets), _ptr(a), _ld(a), _ptr(sa), _ld(sa), _ptr(b),
                                        _ptr(sb), act, _ptr(d), _ld(d), out_dtype, _ptr(gu),
                                        _ld(gu) if gu is not None else 0, accum, _stream()), "fp8_grouped_gated_gemm")
    return d, gu


def fp8_grouped_gated_gemm_quant(offsets, a, sa, b, sb, act=ACT_SILU, scale_mode=SCALE_FP32, rows_bound=None, q=None,
                                 s=None, gu=None, save_gu=False, accum=ACCUM_FP32):
    """fp8_gated_gemm_quant over experts; returns (q, s, gu or None)."""
    M, N, K, G = _gated_operands(a, sa, b, sb, accum, rows_bound, offsets)
    q, s = _quant_out(q, s, M, N, a, M)
    gu = _gated_kept(gu, save_gu, M, N, a)
    _check(lib().fp8_grouped_gated_gemm_quant(G, M, N, K, _ptr(offsets), _ptr(a), _ld(a), _ptr(sa), _ld(sa), _ptr(b),
                                              _ptr(sb), act, scale_mode, _ptr(q), _ld(q), _ptr(s), _ld(s), _ptr(gu),
                                              _ld(gu) if gu is not None else 0, accum, _stream()),
           "fp8_grouped_gated_gemm_quant")
    return q, s, gu


def _gated_backward(name, lead, P, dh, gu, act, scale_mode, qr, sr, qc, sc, qh, sh, with_rows, with_cols, with_h):
    _need(dh, "dh", BF16, None, None)
    M, N = dh.shape
    _need(gu, "gu", BF16, M, 2 * N)
    args = []
    for on, q, s, qn, sn, qshape, sshape in (
            (with_rows, qr, sr, "qr", "sr", (M, 2 * N), (2 * N // 128, M)),
            (with_cols, qc, sc, "qc", "sc", (2 * N, P), (P // 128, 2 * N)),
            (with_h, qh, sh, "qh", "sh", (N, P), (P // 128, N))):
        if not on:
            args.append((None, None))
            continue
        if q is None:
            q = _new(qshape, U8, dh)
        if s is None:
            s = _new(sshape, F32, dh)
        _need(q, qn, U8, qshape[0], None)
        _need(s, sn, F32, sshape[0], None)
        if q.shape[1] < qshape[1] or s.shape[1] < sshape[1]:
            raise ValueError(f"{qn} and {sn} need {qshape} and {sshape}, got {tuple(q.shape)} and {tuple(s.shape)}")
        args.append((q, s))
    flat = []
    for q, s in args:
        flat += [_ptr(q), _ld(q) if q is not None else 0, _ptr(s), _ld(s) if s is not None else 0]
    _check(getattr(lib(), name)(*lead, M, N, _ptr(dh), _ld(dh), _ptr(gu), _ld(gu), act, scale_mode, *flat, _stream()),
           name)
    return tuple(t for pair in args for t in pair)


def fp8_gated_backward(dh, gu, act=ACT_SILU, scale_mode=SCALE_FP32, qr=None, sr=None, qc=None, sc=None, qh=None,
                       sh=None, with_rows=True, with_cols=True, with_h=True):
    """Backward of the gated product from dh [M, N] and the kept gu [M, 2N]
    (bf16).  Returns (qr, sr, qc, sc, qh, sh): dG | dU in 1x128 groups
    [M, 2N], in 128x1 groups [2N, P] and H in 128x1 groups [N, P], P = M
    rounded up to 128; None for those switched off."""
    P = (dh.shape[0] + 127) // 128 * 128
    return _gated_backward("fp8_gated_backward", (), P, dh, gu, act, scale_mode, qr, sr, qc, sc, qh, sh,
                           with_rows, with_cols, with_h)


def fp8_grouped_gated_backward(offsets, dh, gu, act=ACT_SILU, scale_mode=SCALE_FP32, qr=None, sr=None, qc=None,
                               sc=None, qh=None, sh=None, with_rows=True, with_cols=True, with_h=True):
    """fp8_gated_backward over experts: the 128x1 groups start anew at every
    expert, on the padded axis of fp8_quant_tile_grouped_col (P =
    grouped_col_bound(M, G); what lies past the last group is left as it
    is)."""
    _need(offsets, "offsets", I32, None)
    G = offsets.shape[0] - 1
    if G < 0:
        raise ValueError("offsets must have at least one entry")
    P = grouped_col_bound(dh.shape[0], G)
    return _gated_backward("fp8_grouped_gated_backward", (G, _ptr(offsets)), P, dh, gu, act, scale_mode, qr, sr, qc,
                           sc, qh, sh, with_rows, with_cols, with_h)


# ---- norms ---------------------------------------------------------------------------

NormResidual = collections.namedtuple("NormResidual", "xo h q s rstd_y rstd_x")
NormResidualGrads = collections.namedtuple("NormResidualGrads", "dx dy dw_pre dw_post dgate")


def _seam_inputs(M, D, y, w_post, gate, gate_rows, w_pre):
    if y is not None:
        _need(y, "y", BF16, M, D)
        if y.shape[0] != M:
            raise ValueError(f"y has {y.shape[0]} rows, x has {M}")
    if w_post is not None:
        _need(w_post, "w_post", F32, D)
    if w_pre is not None:
        _need(w_pre, "w_pre", F32, D)
    if gate is None:
        return 0
    rows = max(M, 1) if gate_rows is None else int(gate_rows)
    if rows < 1:
        raise ValueError(f"gate_rows must be at least 1, got {rows}")
    _need(gate, "gate", F32, (M + rows - 1) // rows, D)
    if not gate.is_contiguous():
        raise ValueError("gate must be contiguous")
    return rows


def fp8_norm_residual(x, w_pre=None, y=None, w_post=None, gate=None, gate_rows=None, alpha=1.0, eps=1e-6,
                      scale_mode=SCALE_FP32, quantise=True, want_h=False, xo=None, q=None, s=None, h=None):
    """x' = alpha x + gate * (RMSNorm(y) w_post), then RMSNorm(x') w_pre,
    quantised 1x128 (quantise) and / or in bf16 (want_h).  x, y bf16 [M, D];
    w_pre, w_post fp32 [D]; gate fp32 [ceil(M/gate_rows), D] (gate_rows None:
    one row for all).  Returns NormResidual(xo, h, q, s, rstd_y, rstd_x), None
    for what was not asked for."""
    _need(x, "x", BF16, None, None)
    M, D = x.shape
    rows = _seam_inputs(M, D, y, w_post, gate, gate_rows, w_pre)
    quantise = w_pre is not None and (quantise or q is not None)
    if y is not None:
        if xo is None:
            xo = _new((M, D), BF16, x)
        else:
            _need(xo, "xo", BF16, M, D)
    if quantise:
        q, s = _quant_out(q, s, M, D, x, M)
    if want_h and h is None:
        h = _new((M, D), BF16, x)
    if h is not None:
        _need(h, "h", BF16, M, D)
    ry = _new((M,), F32, x) if w_post is not None else None
    rx = _new((M,), F32, x) if w_pre is not None else None
    _check(lib().fp8_norm_residual(M, D, _ptr(x), _ld(x), _ptr(y), _ld(y) if y is not None else 0, _ptr(w_post),
                                   _ptr(gate), rows, alpha, eps, _ptr(xo), _ld(xo) if xo is not None else 0,
                                   _ptr(w_pre), _ptr(h), _ld(h) if h is not None else 0, scale_mode, _ptr(q),
                                   _ld(q) if q is not None else 0, _ptr(s), _ld(s) if s is not None else 0, _ptr(ry),
                                   _ptr(rx), _stream()), "fp8_norm_residual")
    return NormResidual(xo, h, q, s, ry, rx)


def fp8_norm_residual_backward(dxo, dh, xo, rstd_x, w_pre, y=None, rstd_y=None, w_post=None, gate=None,
                               gate_rows=None, alpha=1.0, dx=None, dy=None, workspace=None):
    """Gradients of fp8_norm_residual from dxo (of x', or None) and dh (of
    RMSNorm(x') w_pre, or None), bf16 [M, D].  Returns NormResidualGrads(dx,
    dy, dw_pre, dw_post, dgate), None where the input was None."""
    lead = dxo if dxo is not None else dh
    _need(lead, "dxo" if dxo is not None else "dh", BF16, None, None)
    M, D = lead.shape
    if dh is not None:
        for t, name in ((dh, "dh"), (xo, "xo")):
            _need(t, name, BF16, M, D)
        _need(rstd_x, "rstd_x", F32, M)
        _need(w_pre, "w_pre", F32, D)
    rows = _seam_inputs(M, D, y, w_post, gate, gate_rows, None)
    if w_post is not None:
        _need(rstd_y, "rstd_y", F32, M)
    if dx is None:
        dx = _new((M, D), BF16, lead)
    else:
        _need(dx, "dx", BF16, M, D)
    if y is not None:
        if dy is None:
            dy = _new((M, D), BF16, lead)
        else:
            _need(dy, "dy", BF16, M, D)
    dw_pre = _new((D,), F32, lead) if dh is not None else None
    dw_post = _new((D,), F32, lead) if w_post is not None else None
    dgate = torch.empty_like(gate) if gate is not None else None
    need = int(lib().fp8_norm_backward_workspace_bytes(M, D))
    if workspace is None:
        workspace = _new((need,), U8, lead)
    _need(workspace, "workspace", U8, None)
    ld = lambda t: _ld(t) if t is not None else 0  # noqa: E731
    _check(lib().fp8_norm_residual_backward(
        M, D, _ptr(dxo), ld(dxo), _ptr(dh), ld(dh), _ptr(xo) if dh is not None else None, ld(xo) if dh is not None else 0,
        _ptr(rstd_x) if dh is not None else None, _ptr(w_pre) if dh is not None else None, _ptr(y), ld(y),
        _ptr(rstd_y) if w_post is not None else None, _ptr(w_post), _ptr(gate), rows, alpha, _ptr(dx), ld(dx), _ptr(dy),
        ld(dy), _ptr(dw_pre), _ptr(dw_post), _ptr(dgate), _ptr(workspace), workspace.numel(), _stream()),
        "fp8_norm_residual_backward")
    return NormResidualGrads(dx, dy, dw_pre, dw_post, dgate)


# ---- gradient norm and clipping -------------------------------------------------------

def _grad_table(grads, name):
    """(pointers, counts, types) as host arrays of the C ABI."""
    n = len(grads)
    ptr, count, dtype = (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)(), (ctypes.c_int32 * n)()
    here = torch.cuda.current_device()
    for i, g in enumerate(grads):
        if not isinstance(g, torch.Tensor) or not g.is_cuda or g.get_device() != here:
            raise TypeError(f"{name}[{i}] must be a CUDA (HIP) tensor on the current device")
        if g.dtype is not F32 and g.dtype is not BF16:
            raise TypeError(f"{name}[{i}] must be float32 or bfloat16, got {g.dtype}")
        if not g.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous")
        ptr[i], count[i], dtype[i] = g.data_ptr(), g.numel(), OUT_F32 if g.dtype is F32 else OUT_BF16
    return ptr, count, dtype


def _grad_workspace(n, workspace):
    need = int(lib().fp8_grad_workspace_bytes(n))
    if workspace is None:
        workspace = torch.empty(need, dtype=U8, device="cuda")
    _need(workspace, "workspace", U8, None)
    return workspace


def fp8_grad_norm(grads, workspace=None):
    """The 2-norm of all gradients together (fp32 or bf16, any sizes): a
    one-element fp32 tensor on the device."""
    grads = list(grads)
    ptr, count, dtype = _grad_table(grads, "grads")
    ws = _grad_workspace(len(grads), workspace)
    norm = torch.empty(1, dtype=F32, device="cuda")
    _check(lib().fp8_grad_norm(len(grads), ptr, count, dtype, _ptr(norm), _ptr(ws), ws.numel(), _stream()),
           "fp8_grad_norm")
    return norm


def fp8_grad_clip(grads, max_norm, out=None, workspace=None):
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place or
    into `out` (tensors of the same types and sizes).  Returns (norm, coef),
    one-element fp32 tensors on the device."""
    grads = list(grads)
    out = grads if out is None else list(out)
    ptr, count, dtype = _grad_table(grads, "grads")
    optr, ocount, odtype = (ptr, count, dtype) if out is grads else _grad_table(out, "out")
    if len(out) != len(grads) or list(ocount) != list(count) or list(odtype) != list(dtype):
        raise ValueError("out must match grads in number, sizes and types")
    ws = _grad_workspace(len(grads), workspace)
    res = torch.empty(2, dtype=F32, device="cuda")
    norm, coef = res[:1], res[1:]
    _check(lib().fp8_grad_clip(len(grads), ptr, count, dtype, float(max_norm), optr, _ptr(norm), _ptr(coef), _ptr(ws),
                               ws.numel(), _stream()), "fp8_grad_clip")
    return norm, coef
