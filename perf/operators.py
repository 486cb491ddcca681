"""Measured cases of the feed-forward block's operators around the FP8 GEMMs.

Each operator is written here twice: in plain torch operations in 32 bits
(`own = False`) and as the calls of this package (`own = True`).  `exact`
computes the same from the definitions in 64 bits.

The operators:
  gated     H = act(X Wg^T) * (X Wu^T) from FP8 codes and their scales, with
            the pre-activations kept for the backward pass where asked;
            dense, or grouped over MoE experts
  gated_bwd from dH and the kept pre-activations: the gradients of both
            projections' outputs, quantised 1x128 (for Dgrad) and 128x1 (for
            Wgrad), and H again, quantised 128x1 (for the next Wgrad)
  norm      x' = alpha x + gate * RMSNorm(y) w_post, then RMSNorm(x') w_pre
            quantised 1x128: the seam between two blocks
  norm_bwd  its gradients
  clip      the global norm of many gradients, and the gradients clipped by it
"""
import math

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 448.0 * 2.0 ** -126
EPS = 1e-6


# ---- cases -------------------------------------------------------------------------

def listed():
    return [
        # one token through a shared expert while serving: the latency of one call
        dict(name="gated one token", op="gated", G=0, M=1, N=2048, K=7168, act="silu", out="bf16", accum="mfma8",
             save=False, rows="even"),
        # the dense feed-forward layer of a training step, pre-activations kept
        dict(name="gated training", op="gated", G=0, M=4096, N=18432, K=7168, act="silu", out="bf16",
             accum="mfma8", save=True, rows="even"),
        # a prompt's tokens over 32 experts, about 128 rows each
        dict(name="gated experts prompt", op="gated", G=32, M=4096, N=2048, K=7168, act="silu", out="bf16",
             accum="mfma8_pow2", save=False, rows="uneven"),
        # a decoding batch over 64 experts, some of them without a token; exact
        # sums, H leaves quantised for the down-projection
        dict(name="gated experts decode", op="gated", G=64, M=509, N=2048, K=7168, act="silu", out="quant",
             accum="fp32", save=False, rows="uneven"),
        # the backward pass of the dense layer
        dict(name="gated backward training", op="gated_bwd", G=0, M=4096, N=18432, act="silu", rows="even"),
        # the backward pass of 32 experts with uneven rows
        dict(name="gated backward experts", op="gated_bwd", G=32, M=4103, N=2048, act="gelu", rows="uneven"),
        # the seam between two blocks for one token
        dict(name="norm one token", op="norm", M=1, D=7168, post=True, gate_rows=1, alpha=1.0),
        # the same for a training batch, a gate for each of its sequences
        dict(name="norm training", op="norm", M=8192, D=7168, post=True, gate_rows=2048, alpha=1.0),
        # its backward pass
        dict(name="norm backward training", op="norm_bwd", M=8192, D=7168, post=True, gate_rows=2048, alpha=1.0),
        # a short ragged batch: the sequences' length does not divide the rows
        dict(name="norm backward ragged", op="norm_bwd", M=333, D=2048, post=True, gate_rows=100, alpha=0.5),
        # the small parameters of a model: norms, biases, routers
        dict(name="clip small tensors", op="clip", n=48, largest=60000, dtype="mixed", spread=True),
        # the FP32 weight gradients of 32 experts' stacked gate and up projections
        dict(name="clip expert gradients", op="clip", n=32, largest=4096 * 7168, dtype="fp32", spread=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_bwd", "norm", "norm_bwd", "clip"])
    if op == "gated":
        out, accum = rng.choice([("bf16", "mfma8"), ("bf16", "mfma8_pow2"), ("f32", "fp32"), ("quant", "fp32")])
        G = rng.choice([0, 0, 1, 8, 32, 64])
        K = 128 * _log_int(rng, 1, 56)
        N = 128 * _log_int(rng, 1, 16 if G else 144)
        return dict(op=op, G=G, M=_log_int(rng, 1, 4096), N=N, K=K, act=rng.choice(["silu", "gelu"]), out=out,
                    accum=accum, save=rng.random() < 0.5, rows="uneven" if G else "even")
    if op == "gated_bwd":
        G = rng.choice([0, 1, 8, 32, 64])
        return dict(op=op, G=G, M=_log_int(rng, 1, 4096), N=128 * _log_int(rng, 1, 144),
                    act=rng.choice(["silu", "gelu"]), rows="uneven" if G else "even")
    if op in ("norm", "norm_bwd"):
        M = _log_int(rng, 1, 8192)
        return dict(op=op, M=M, D=128 * rng.randint(1, 64), post=rng.random() < 0.8,
                    gate_rows=_log_int(rng, 1, M), alpha=rng.choice([1.0, 0.5, 1.4142135]))
    return dict(op=op, n=rng.randint(1, 40), largest=_log_int(rng, 1, 8_000_000),
                dtype=rng.choice(["fp32", "bf16", "mixed"]), spread=rng.random() < 0.7)


# ---- inputs ------------------------------------------------------------------------

def _decode(q):
    """The values of E4M3 codes held as uint8."""
    return q.view(torch.float8_e4m3fn)


def _scale(amax, pow2):
    amax = amax.clamp_min(AMAX_FLOOR)
    if not pow2:
        return amax / E4M3_MAX
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 1.75 * 2^8
    return torch.ldexp(torch.ones_like(amax), e - 9 + (m > 0.875).to(e.dtype))


def _codes(x, s):
    return (x / s).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _make_rows(gen, M, K, pow2):
    """Activation codes [M, K] and scales [K/128, M]: normal values with a few outliers."""
    x = torch.randn(M, K, generator=gen, device="cuda")
    x = x * torch.where(torch.rand(M, K, generator=gen, device="cuda") < 1e-3, 100.0, 1.0)
    g = x.view(M, K // 128, 128)
    s = _scale(g.abs().amax(2), pow2)
    return _codes(g, s[:, :, None]).view(M, K), s.t().contiguous()


def _make_weight(gen, R, K, pow2):
    """Weight codes [R, K] and scales [R/128, K/128]."""
    w = torch.randn(R, K, generator=gen, device="cuda") * 0.02
    b = w.view(R // 128, 128, K // 128, 128)
    s = _scale(b.abs().amax((1, 3)), pow2)
    return _codes(b, s[:, None, :, None]).view(R, K), s


def _make_offsets(case, gen):
    """Row ranges of the experts: uneven, some experts empty."""
    G, M = case["G"], case["M"]
    share = torch.rand(G, generator=gen, device="cuda", dtype=torch.float64) ** 2
    share = share * (torch.rand(G, generator=gen, device="cuda") > 0.1) + 1e-9
    ends = torch.round(share.cumsum(0) / share.sum() * M).to(torch.int32)
    ends[-1] = M
    off = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), ends])
    return off


def _clip_sizes(case):
    """The tensors' element counts: all alike, or spread over the logarithm from 1 to the largest."""
    n, top = case["n"], case["largest"]
    if not case["spread"]:
        return [top] * n
    return [max(1, int(round(top ** (1 - (0.618034 * i) % 1)))) for i in range(n)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    st = dict(case)
    if op == "gated":
        pow2 = case["accum"] == "mfma8_pow2"
        G, M, N, K = case["G"], case["M"], case["N"], case["K"]
        st["qx"], st["sx"] = _make_rows(gen, M, K, pow2)
        parts = [_make_weight(gen, 2 * N, K, pow2) for _ in range(max(1, G))]
        if G:
            st["offsets"] = _make_offsets(case, gen)
            st["qw"] = torch.stack([p[0] for p in parts])
            st["sw"] = torch.stack([p[1] for p in parts])
            st["longest"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())
        else:
            st["qw"], st["sw"] = parts[0]
    elif op == "gated_bwd":
        M, N, G = case["M"], case["N"], case["G"]
        st["gu"] = (torch.randn(M, 2 * N, generator=gen, device="cuda") * 1.5).bfloat16()
        st["dh"] = (torch.randn(M, N, generator=gen, device="cuda") * 1e-3).bfloat16()
        if G:
            st["offsets"] = _make_offsets(case, gen)
        # the padded token axis of the 128x1 groups, zero where no group reaches
        P = 128 * ((M + 127) // 128 + G)
        st["qc"] = torch.zeros(2 * N, P, dtype=torch.uint8, device="cuda")
        st["sc"] = torch.zeros(P // 128, 2 * N, device="cuda")
        st["qh"] = torch.zeros(N, P, dtype=torch.uint8, device="cuda")
        st["sh"] = torch.zeros(P // 128, N, device="cuda")
    elif op in ("norm", "norm_bwd"):
        M, D = case["M"], case["D"]
        B = -(-M // case["gate_rows"])
        st["x"] = torch.randn(M, D, generator=gen, device="cuda").bfloat16()
        st["y"] = (torch.randn(M, D, generator=gen, device="cuda") * 3.0).bfloat16()
        st["w_pre"] = 1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")
        st["w_post"] = 1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda") if case["post"] else None
        st["gate"] = torch.randn(B, D, generator=gen, device="cuda") * 0.5
        if op == "norm_bwd":
            xo, st["ry"], st["rx"] = _seam(st)[:3]
            st["xo"] = xo.bfloat16()
            st["dxo"] = torch.randn(M, D, generator=gen, device="cuda").bfloat16()
            st["dh"] = torch.randn(M, D, generator=gen, device="cuda").bfloat16()
            del st["x"]
    else:
        n, sizes = case["n"], _clip_sizes(case)
        kinds = [torch.float32 if case["dtype"] == "fp32" or (case["dtype"] == "mixed" and i % 3) else torch.bfloat16
                 for i in range(n)]
        st["grads"] = [(torch.randn(k, generator=gen, device="cuda") * 1e-2).to(t) for k, t in zip(sizes, kinds)]
        st["out"] = [torch.empty_like(g) for g in st["grads"]]
    return st


# ---- plain forms -------------------------------------------------------------------

def _act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _rows32(q, s):
    M, K = q.shape
    return (_decode(q).float().view(M, K // 128, 128) * s.t()[:, :, None]).view(M, K)


def _weight32(q, s):
    *lead, R, K = q.shape
    w = _decode(q).float().view(*lead, R // 128, 128, K // 128, 128)
    return (w * s[..., :, None, :, None]).view(*lead, R, K)


def _quant_rows(x):
    """1x128 groups: codes [M, C], scales [C/128, M]."""
    M, C = x.shape
    g = x.view(M, C // 128, 128)
    amax = g.abs().amax(2).clamp_min(AMAX_FLOOR)
    q = (g * (E4M3_MAX / amax)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(M, C), (amax / E4M3_MAX).t().contiguous()


def _quant_cols(x):
    """128x1 groups of a row count that is a multiple of 128: codes [C, P], scales [P/128, C]."""
    q, s = _quant_rows(x.t().contiguous())
    return q, s


def _ranks(offsets, M):
    """For each of M rows its expert and its place among the expert's rows."""
    r = torch.arange(M, device="cuda")
    e = torch.searchsorted(offsets[1:].contiguous(), r.to(torch.int32), right=True)
    return e, r - offsets[e]


def _gated_plain(st):
    x, w, N = _rows32(st["qx"], st["sx"]), _weight32(st["qw"], st["sw"]), st["N"]
    if st["G"]:
        # rows of each expert side by side, padded to the longest one
        e, i = _ranks(st["offsets"], st["M"])
        pad = x.new_zeros(st["G"], max(1, st["longest"]), st["K"])
        pad[e, i] = x
        gu = torch.bmm(pad, w.transpose(1, 2).contiguous())[e, i]
    else:
        gu = x @ w.t()
    h = _act(gu[:, :N], st["act"])[0] * gu[:, N:]
    kept = {"gu": gu.bfloat16()} if st["save"] else {}
    if st["out"] == "quant":
        q, s = _quant_rows(h)
        return {"q": q, "s": s, **kept}
    return {"h": h.bfloat16() if st["out"] == "bf16" else h, **kept}


def _gated_bwd_plain(st):
    M, N = st["M"], st["N"]
    g, u, dh = st["gu"][:, :N].float(), st["gu"][:, N:].float(), st["dh"].float()
    a, da = _act(g, st["act"])
    dgu = torch.cat([dh * u * da, dh * a], 1)
    qr, sr = _quant_rows(dgu)
    place = torch.arange(M, device="cuda")
    used = (M + 127) // 128
    if st["G"]:
        e, i = _ranks(st["offsets"], M)
        groups = (st["offsets"][1:] - st["offsets"][:-1] + 127) // 128
        place = (groups.cumsum(0) - groups)[e] * 128 + i
        used = groups.sum()
    reach = torch.arange(st["sc"].shape[0], device="cuda") < used  # the groups that hold a row
    both = torch.zeros(st["qc"].shape[1], 3 * N, device="cuda")
    both[place] = torch.cat([dgu, a * u], 1)
    q, s = _quant_cols(both)
    s = torch.where(reach[:, None], s, torch.zeros_like(s))
    return {"qr": qr, "sr": sr, "qc": q[: 2 * N], "sc": s[:, : 2 * N].contiguous(), "qh": q[2 * N:],
            "sh": s[:, 2 * N:].contiguous()}


def _gate_of(st, M):
    return st["gate"][torch.arange(M, device="cuda") // st["gate_rows"]]


def _seam(st):
    x, y = st["x"].float(), st["y"].float()
    ry = torch.rsqrt(y.square().mean(1) + EPS)
    n = y * ry[:, None] * st["w_post"] if st["post"] else y
    xo = st["alpha"] * x + _gate_of(st, x.shape[0]) * n
    rx = torch.rsqrt(xo.square().mean(1) + EPS)
    return xo, ry, rx, xo * rx[:, None] * st["w_pre"]


def _norm_plain(st):
    xo, ry, rx, h = _seam(st)
    q, s = _quant_rows(h)
    kept = {"ry": ry} if st["post"] else {}
    return {"xo": xo.bfloat16(), "q": q, "s": s, "rx": rx, **kept}


def _norm_bwd_plain(st):
    M, D = st["xo"].shape
    xo, y, dh, t = st["xo"].float(), st["y"].float(), st["dh"].float(), st["dxo"].float()
    rx, ry, gate = st["rx"][:, None], st["ry"][:, None], _gate_of(st, M)
    v = dh * st["w_pre"]
    t = t + rx * v - xo * rx ** 3 * (v * xo).mean(1, keepdim=True)
    dw_pre = (dh * xo * rx).sum(0)
    dn = gate * t
    yhat = y * ry if st["post"] else y
    n = yhat * st["w_post"] if st["post"] else y
    B, gr = st["gate"].shape[0], st["gate_rows"]
    per = torch.zeros(B * gr, D, device="cuda")
    per[:M] = t * n
    got = {"dx": (st["alpha"] * t).bfloat16(), "dw_pre": dw_pre, "dgate": per.view(B, gr, D).sum(1)}
    if st["post"]:
        z = dn * st["w_post"]
        got["dw_post"] = (dn * yhat).sum(0)
        dn = ry * z - y * ry ** 3 * (z * y).mean(1, keepdim=True)
    got["dy"] = dn.bfloat16()
    return got


def _clip_plain(st):
    total = torch.stack([g.double().square().sum() for g in st["grads"]]).sum().sqrt()
    coef = (1.0 / (total + 1e-6)).clamp_max(1.0).float()
    return {"norm": total.float().view(1), "coef": coef.view(1),
            "grads": [(g.float() * coef).to(g.dtype) for g in st["grads"]]}


# ---- the framework's calls ---------------------------------------------------------

def _bs():
    import block_scaled_gemm_amd
    return block_scaled_gemm_amd


def _gated_own(st):
    bs = _bs()
    act = bs.ACT_SILU if st["act"] == "silu" else bs.ACT_GELU
    accum = {"fp32": bs.ACCUM_FP32, "mfma8": bs.ACCUM_MFMA8, "mfma8_pow2": bs.ACCUM_MFMA8_POW2}[st["accum"]]
    args = (st["qx"], st["sx"], st["qw"], st["sw"], act)
    if st["out"] == "quant":
        if st["G"]:
            q, s, gu = bs.fp8_grouped_gated_gemm_quant(st["offsets"], *args, bs.SCALE_FP32, save_gu=st["save"],
                                                       accum=accum)
        else:
            q, s, gu = bs.fp8_gated_gemm_quant(*args, bs.SCALE_FP32, save_gu=st["save"], accum=accum)
        return {"q": _decode(q), "s": s, **({"gu": gu} if st["save"] else {})}
    out = bs.OUT_BF16 if st["out"] == "bf16" else bs.OUT_F32
    if st["G"]:
        h, gu = bs.fp8_grouped_gated_gemm(st["offsets"], *args, out, save_gu=st["save"], accum=accum)
    else:
        h, gu = bs.fp8_gated_gemm(*args, out, save_gu=st["save"], accum=accum)
    return {"h": h, **({"gu": gu} if st["save"] else {})}


def _gated_bwd_own(st):
    bs = _bs()
    act = bs.ACT_SILU if st["act"] == "silu" else bs.ACT_GELU
    into = dict(qc=st["qc"], sc=st["sc"], qh=st["qh"], sh=st["sh"])
    if st["G"]:
        qr, sr, qc, sc, qh, sh = bs.fp8_grouped_gated_backward(st["offsets"], st["dh"], st["gu"], act, bs.SCALE_FP32,
                                                               **into)
    else:
        qr, sr, qc, sc, qh, sh = bs.fp8_gated_backward(st["dh"], st["gu"], act, bs.SCALE_FP32, **into)
    return {"qr": _decode(qr), "sr": sr, "qc": _decode(qc), "sc": sc, "qh": _decode(qh), "sh": sh}


def _norm_own(st):
    r = _bs().fp8_norm_residual(st["x"], st["w_pre"], y=st["y"], w_post=st["w_post"], gate=st["gate"],
                                gate_rows=st["gate_rows"], alpha=st["alpha"], eps=EPS)
    kept = {"ry": r.rstd_y} if st["post"] else {}
    return {"xo": r.xo, "q": _decode(r.q), "s": r.s, "rx": r.rstd_x, **kept}


def _norm_bwd_own(st):
    r = _bs().fp8_norm_residual_backward(st["dxo"], st["dh"], st["xo"], st["rx"], st["w_pre"], y=st["y"],
                                         rstd_y=st["ry"] if st["post"] else None, w_post=st["w_post"],
                                         gate=st["gate"], gate_rows=st["gate_rows"], alpha=st["alpha"])
    got = {"dx": r.dx, "dw_pre": r.dw_pre, "dgate": r.dgate, "dy": r.dy}
    return {**got, "dw_post": r.dw_post} if st["post"] else got


def _clip_own(st):
    norm, coef = _bs().fp8_grad_clip(st["grads"], 1.0, out=st["out"])
    return {"norm": norm, "coef": coef, "grads": st["out"]}


def run(state):
    op = state["op"]
    if own:
        return {"gated": _gated_own, "gated_bwd": _gated_bwd_own, "norm": _norm_own, "norm_bwd": _norm_bwd_own,
                "clip": _clip_own}[op](state)
    return {"gated": _gated_plain, "gated_bwd": _gated_bwd_plain, "norm": _norm_plain, "norm_bwd": _norm_bwd_plain,
            "clip": _clip_plain}[op](state)


# ---- work --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "gated":
        G, M, N, K = max(1, case["G"]), case["M"], case["N"], case["K"]
        # at most as many experts as rows have anything to multiply
        used = min(G, M)
        read = M * K + 4 * M * K / 128 + used * (2 * N * K + 4 * 2 * N * K / 128 / 128)
        out = {"bf16": 2.0, "f32": 4.0, "quant": 1 + 4 / 128}[case["out"]] + (4.0 if case["save"] else 0.0)
        return {"bytes": read + out * M * N, "flops": 4.0 * M * N * K}
    if op == "gated_bwd":
        M, N = case["M"], case["N"]
        return {"bytes": M * N * (6 + 5 * (1 + 4 / 128)), "flops": 30.0 * M * N}
    if op in ("norm", "norm_bwd"):
        M, D = case["M"], case["D"]
        B = -(-M // case["gate_rows"])
        small = 4 * D * (1 + (1 if case["post"] else 0) + B)
        if op == "norm":
            return {"bytes": M * D * (6 + 1 + 4 / 128) + 8 * M + small, "flops": 12.0 * M * D}
        return {"bytes": M * D * 12 + 8 * M + 2 * small, "flops": 30.0 * M * D}
    sizes = _clip_sizes(case)
    size = [4 if case["dtype"] == "fp32" or (case["dtype"] == "mixed" and i % 3) else 2 for i in range(case["n"])]
    return {"bytes": 2.0 * sum(k * b for k, b in zip(sizes, size)), "flops": 3.0 * sum(sizes)}


# ---- 64 bits -----------------------------------------------------------------------

def _value64(q):
    return q.view(torch.float8_e4m3fn).to(torch.float64)


def _sigmoid64(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _act64(g, kind):
    # both are g * sigmoid(p(g)); the derivative follows from the product rule
    if kind == "silu":
        p, dp = g, torch.ones_like(g)
    else:
        k = 2.0 * math.sqrt(2.0 / math.pi)
        p, dp = k * (g + 0.044715 * g ** 3), k * (1 + 3 * 0.044715 * g ** 2)
    s = _sigmoid64(p)
    return g * s, s + g * s * (1 - s) * dp


def _groups64(x):
    """x [M, C] in 1x128 groups: the values of the codes and the scales [C/128, M]."""
    M, C = x.shape
    g = x.reshape(M, C // 128, 128)
    s = torch.clamp(g.abs().max(2).values, min=AMAX_FLOOR) / E4M3_MAX
    v = (g / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).reshape(M, C), s.t().contiguous()


def _exact_gated(st):
    M, N, K = st["M"], st["N"], st["K"]
    x = _value64(st["qx"]) * st["sx"].double().repeat_interleave(128, 0).t()
    gu = torch.empty(M, 2 * N, dtype=torch.float64, device="cuda")
    bounds = st["offsets"].tolist() if st["G"] else [0, M]
    qw, sw = (st["qw"], st["sw"]) if st["G"] else (st["qw"][None], st["sw"][None])
    for e in range(len(bounds) - 1):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            w = _value64(qw[e]) * sw[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            gu[lo:hi] = x[lo:hi] @ w.t()
    h = _act64(gu[:, :N], st["act"])[0] * gu[:, N:]
    kept = {"gu": gu} if st["save"] else {}
    if st["out"] == "quant":
        q, s = _groups64(h)
        return {"q": q, "s": s, **kept}
    return {"h": h, **kept}


def _exact_gated_bwd(st):
    M, N, P = st["M"], st["N"], st["qc"].shape[1]
    bounds = st["offsets"].tolist() if st["G"] else [0, M]
    q = torch.zeros(3 * N, P, dtype=torch.float64, device="cuda")
    s = torch.zeros(P // 128, 3 * N, dtype=torch.float64, device="cuda")
    qr = torch.empty(M, 2 * N, dtype=torch.float64, device="cuda")
    sr = torch.empty(2 * N // 128, M, dtype=torch.float64, device="cuda")
    at = 0
    for e in range(len(bounds) - 1):
        for lo in range(bounds[e], bounds[e + 1], 128):
            hi = min(lo + 128, bounds[e + 1])
            g, u = st["gu"][lo:hi, :N].double(), st["gu"][lo:hi, N:].double()
            dh = st["dh"][lo:hi].double()
            a, da = _act64(g, st["act"])
            both = torch.cat([dh * u * da, dh * a, a * u], 1)
            qr[lo:hi], sr[:, lo:hi] = _groups64(both[:, : 2 * N])
            full = torch.zeros(128, 3 * N, dtype=torch.float64, device="cuda")
            full[: hi - lo] = both
            q[:, at:at + 128], srow = _groups64(full.t())
            s[at // 128] = srow[0]
            at += 128
    return {"qr": qr, "sr": sr, "qc": q[: 2 * N], "sc": s[:, : 2 * N].contiguous(), "qh": q[2 * N:],
            "sh": s[:, 2 * N:].contiguous()}


def _exact_norm(st):
    x, y = st["x"].double(), st["y"].double()
    M, D = x.shape
    gate = st["gate"].double().repeat_interleave(st["gate_rows"], 0)[:M]
    ry = (y.pow(2).sum(1) / D + EPS) ** -0.5
    n = y * ry[:, None] * st["w_post"].double() if st["post"] else y
    xo = x * st["alpha"] + n * gate
    rx = (xo.pow(2).sum(1) / D + EPS) ** -0.5
    q, s = _groups64(xo * rx[:, None] * st["w_pre"].double())
    return {"xo": xo, "q": q, "s": s, "rx": rx, **({"ry": ry} if st["post"] else {})}


def _exact_norm_bwd(st):
    # by torch's differentiation of the plain definition, with the saved
    # statistics standing for those of the saved rows
    M, D = st["xo"].shape
    xo, y, dh, dxo = (st[k].double() for k in ("xo", "y", "dh", "dxo"))
    rx = st["rx"].double()[:, None]
    xhat = xo * rx
    v = dh * st["w_pre"].double()
    t = dxo + rx * (v - xhat * ((v * xhat).sum(1, keepdim=True) / D))
    gate = st["gate"].double().repeat_interleave(st["gate_rows"], 0)[:M]
    got = {"dx": t * st["alpha"], "dw_pre": torch.einsum("md,md->d", dh, xhat)}
    dn = t * gate
    if st["post"]:
        ry, wp = st["ry"].double()[:, None], st["w_post"].double()
        yhat = y * ry
        z = dn * wp
        got["dw_post"] = torch.einsum("md,md->d", dn, yhat)
        got["dy"] = ry * (z - yhat * ((z * yhat).sum(1, keepdim=True) / D))
        n = yhat * wp
    else:
        got["dy"] = dn
        n = y
    rows = torch.arange(M, device="cuda") // st["gate_rows"]
    got["dgate"] = torch.zeros(st["gate"].shape, dtype=torch.float64, device="cuda").index_add_(0, rows, t * n)
    return got


def _exact_clip(st):
    total = math.sqrt(math.fsum(float(g.double().norm()) ** 2 for g in st["grads"]))
    coef = min(1.0, 1.0 / (total + 1e-6))
    one = dict(dtype=torch.float64, device="cuda")
    return {"norm": torch.tensor([total], **one), "coef": torch.tensor([coef], **one),
            "grads": [g.double() * coef for g in st["grads"]]}


def exact(case, seed):
    st = prepare(case, seed)
    return {"gated": _exact_gated, "gated_bwd": _exact_gated_bwd, "norm": _exact_norm, "norm_bwd": _exact_norm_bwd,
            "clip": _exact_clip}[case["op"]](st)
