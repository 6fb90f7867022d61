"""What is measured of the operators of an 8-bit training step between its products: layer norm with its
gradients, the gated activation with its gradients, activation checkpoints as E4M3 codes with a scale per
block of 128, and what a backward pass makes of such checkpoints.

`run` is one pass through an operator. With `own` it makes the calls a user makes of
mx_microscaling_quantize_gb300; without, it computes the same in elementary torch operations in 32
bits. `exact` computes it from the definition in 64 bits."""

import math

import torch

own = False

DEV = "cuda"
BLK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # blocks below this abs-max are scaled as if it were their abs-max
EPS = 1e-5


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a serving step on its way into an 8-bit product
        dict(name="norm_one_token", op="norm", M=1, K=8192, dtype="bf16", out="codes", center=True),
        # a prompt's residual stream, kept in fp32, normalised to bf16
        dict(name="norm_prompt", op="norm", M=8192, K=8192, dtype="fp32", out="bf16", center=True),
        # a training step on a ragged batch, nothing in 8 bits
        dict(name="norm_train_ragged", op="norm_train", M=4001, K=2048, dtype="bf16",
             checkpoint=False, center=True),
        # a training step that keeps the residual stream in 8 bits and feeds an 8-bit product
        dict(name="norm_train_checkpoint", op="norm_train", M=8192, K=8192, dtype="bf16",
             checkpoint=True, center=True),
        # 16 tokens of a serving step in 8 experts each
        dict(name="act_decode", op="act", R=128, H=1024, kind="silu", gated=True),
        # a prompt of 4096 tokens through the widest layer of the library's workloads
        dict(name="act_prompt", op="act", R=4096, H=28672, kind="silu", gated=True),
        # a training step's expert rows: forward, and backward from the checkpoint
        dict(name="act_train_experts", op="act_train", R=16384, H=1024, kind="silu", gated=True),
        # the same of the widest layer
        dict(name="act_train_wide", op="act_train", R=4096, H=28672, kind="silu", gated=True),
        # 16384 expert rows gathered from 4096 checkpointed tokens, for the weights' gradient
        dict(name="cols_experts", op="cols", M=4096, K=2048, k=4, E=128, skew=1.1),
        # a large dense layer's checkpoint, for the weights' gradient
        dict(name="cols_large", op="cols", M=8192, K=8192, k=0, E=1, skew=0.0),
        # the smallest activation of the library's workloads back from its checkpoint
        dict(name="dequantize_small", op="dequantize", M=128, K=4096, R=0, out="bf16"),
        # a large one
        dict(name="dequantize_large", op="dequantize", M=8192, K=8192, R=0, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_train", "act", "act_train", "cols", "dequantize"))
    dtype = rng.choice(("bf16", "bf16", "fp32"))
    if op == "norm":
        out = rng.choice(("bf16", "codes", "fp32"))
        K = 32 * _log(rng, 2, 256) if out == "codes" or rng.random() < 0.5 else _log(rng, 33, 8192)
        return dict(op=op, M=_log(rng, 1, 8192), K=K, dtype=dtype, out=out,
                    center=rng.random() < 0.7)
    if op == "norm_train":
        checkpoint = rng.random() < 0.5
        K = 32 * _log(rng, 2, 256) if checkpoint or rng.random() < 0.7 else _log(rng, 33, 8192)
        return dict(op=op, M=_log(rng, 1, 8192), K=K, dtype=dtype, checkpoint=checkpoint,
                    center=rng.random() < 0.7)
    if op in ("act", "act_train"):
        gated = rng.random() < 0.7
        step, most = (128, 224) if op == "act_train" and gated else (32, 896)
        return dict(op=op, R=_log(rng, 1, 4096), H=step * _log(rng, 1, most),
                    kind=rng.choice(("silu", "silu", "gelu", "gelu_tanh")), gated=gated)
    if op == "cols":
        if rng.random() < 0.5:
            return dict(op=op, M=_log(rng, 1, 8192), K=32 * _log(rng, 2, 256), k=0, E=1, skew=0.0)
        E = _log(rng, 2, 128)
        k = rng.randint(1, min(8, E))
        return dict(op=op, M=_log(rng, 1, 16384 // k), K=32 * _log(rng, 2, 64), k=k, E=E,
                    skew=rng.choice((0.0, 1.1)))
    R = _log(rng, 1, 8192) if rng.random() < 0.4 else 0
    return dict(op=op, M=_log(rng, 1, 8192), K=32 * _log(rng, 2, 256), R=R,
                out=rng.choice(("bf16", "fp32")))


def work(case):
    op = case["op"]
    sc = 1 + 4 / BLK  # bytes of an element in 8 bits with its share of a scale
    size = {"bf16": 2, "fp32": 4, "codes": sc}
    if op == "norm":
        n = case["M"] * case["K"]
        return {"bytes": n * (size[case["dtype"]] + size[case["out"]]) + 8 * case["K"],
                "flops": 8 * n}
    if op == "norm_train":
        n, x = case["M"] * case["K"], size[case["dtype"]]
        forward = 2 * sc if case["checkpoint"] else 2  # operand and checkpoint, or bf16
        return {"bytes": n * (x + forward + 2 + x) + 8 * case["M"] + 16 * case["K"],
                "flops": 20 * n}
    if op in ("act", "act_train"):
        n, parts = case["R"] * case["H"], 2 if case["gated"] else 1
        if op == "act":
            return {"bytes": n * (2 * parts + sc), "flops": 8 * n}
        # u and dh in; h, the checkpoint, du and its operand out
        return {"bytes": n * (2 * parts + 2 + sc + parts * (sc + 2 + sc)), "flops": 30 * n}
    if op == "cols":
        rows = case["M"] * max(1, case["k"])
        return {"bytes": (case["M"] + rows) * case["K"] * sc, "flops": 4 * rows * case["K"]}
    rows = case["R"] or case["M"]
    return {"bytes": (min(rows, case["M"]) * sc + rows * size[case["out"]]) * case["K"],
            "flops": rows * case["K"]}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _activations(M, K, gen):
    """Normal activations with a few loud channels."""
    x = torch.randn(M, K, generator=gen, device=DEV)
    loud = torch.rand(K, generator=gen, device=DEV) < 0.005
    return x * torch.where(loud, 20.0, 1.0)


def _choices(T, k, E, skew, gen):
    """k distinct experts for each token, by popularity rank^-skew under a random order."""
    logp = -skew * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    logp = logp[torch.randperm(E, generator=gen, device=DEV)]
    u = torch.rand(T, E, generator=gen, device=DEV).clamp_min(1e-12)
    return torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_train"):
        M, K = case["M"], case["K"]
        x = _activations(M, K, gen) + (0.1 + 0.5 * torch.randn(K, generator=gen, device=DEV))
        s["x"] = x.to(_DTYPE[case["dtype"]])
        s["weight"] = 1.0 + 0.1 * torch.randn(K, generator=gen, device=DEV)
        s["bias"] = 0.02 * torch.randn(K, generator=gen, device=DEV) if case["center"] else None
        if op == "norm_train":
            s["dy"] = (torch.randn(M, K, generator=gen, device=DEV) * 1e-3).bfloat16()
        return s
    if op in ("act", "act_train"):
        R, H = case["R"], case["H"]
        s["u"] = _activations(R, H * (2 if case["gated"] else 1), gen).bfloat16()
        if op == "act_train":
            s["dh"] = (torch.randn(R, H, generator=gen, device=DEV) * 1e-3).bfloat16()
        return s
    M, K = case["M"], case["K"]
    s["codes"], s["scales"] = _rows_plain(_activations(M, K, gen).bfloat16())
    if op == "cols":
        s["index"] = s["offsets"] = None
        R, E = M * max(1, case["k"]), case["E"]
        if case["k"]:
            chosen = _choices(M, case["k"], E, case["skew"], gen).flatten()
            s["offsets"] = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
            s["offsets"][1:] = torch.bincount(chosen, minlength=E).cumsum(0)
            s["index"] = (torch.sort(chosen, stable=True).indices // case["k"]).int()
        # what lies past the last expert's columns is the caller's
        P = (R + 127 * E) // BLK * BLK
        s["out_codes"] = torch.zeros(K, P, dtype=torch.uint8, device=DEV)
        s["out_scales"] = torch.zeros(P // BLK, K, device=DEV)
        return s
    s["index"] = None
    if case["R"]:
        s["index"] = torch.randint(0, M, (case["R"],), generator=gen, device=DEV,
                                   dtype=torch.int32)
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _factors(amax):
    a = amax.clamp_min(AMAX_FLOOR)
    return torch.full_like(a, E4M3_MAX) / a, a / E4M3_MAX


def _to_codes(t):
    return t.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _up(n):
    return -(-n // BLK) * BLK


def _rows_plain(x):
    """1 x 128 blocks: codes [R, K] as bytes, scales [ceil(K / 128), R]."""
    R, K = x.shape
    b = torch.nn.functional.pad(x.float(), (0, _up(K) - K)).view(R, -1, BLK)
    r, s = _factors(b.abs().amax(2))
    codes = _to_codes(b * r[:, :, None]).view(R, -1)[:, :K]
    return codes.contiguous(), s.t().contiguous()


def _values(codes, scales):
    """What a checkpoint in the rows form stands for, in 32 bits."""
    v = codes.view(torch.float8_e4m3fn).float()
    return v * scales.t().repeat_interleave(BLK, 1)[:, :v.shape[1]]


def _stands_for(codes):
    return codes.view(torch.float8_e4m3fn)


def _norm_plain(x, weight, bias, center):
    """-> 32-bit y, mean (None unless centred), rstd."""
    v = x.float()
    mean = v.mean(1) if center else None
    if center:
        v = v - mean[:, None]
    rstd = 1.0 / torch.sqrt((v * v).mean(1) + EPS)
    y = v * rstd[:, None] * weight
    return (y if bias is None else y + bias), mean, rstd


def _norm_backward_plain(dy, x, mean, rstd, weight, center):
    """-> 32-bit dx, dweight, dbias (None unless centred)."""
    dy = dy.float()
    xhat = (x - mean[:, None] if center else x) * rstd[:, None]
    g = dy * weight
    dx = g - xhat * (g * xhat).mean(1, keepdim=True)
    if center:
        dx = dx - g.mean(1, keepdim=True)
    return dx * rstd[:, None], (dy * xhat).sum(0), dy.sum(0) if center else None


def _act_plain(g, kind):
    """-> the activation of g and its derivative."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if kind == "gelu":
        p = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(8.0 / math.pi)
    s = 1.0 / (1.0 + torch.exp(-c * (g + 0.044715 * g * g * g)))
    return g * s, s + g * s * (1.0 - s) * c * (1.0 + 3 * 0.044715 * g * g)


def _cols_plain(s):
    """128 x 1 blocks along the (gathered) rows, every expert's rows from a new block on."""
    v = _values(s["codes"], s["scales"])
    R, P = v.shape[0], s["out_codes"].shape[1]
    if s["offsets"] is None:
        v = torch.nn.functional.pad(v, (0, 0, 0, P - R))
    else:
        off = s["offsets"]
        n = off[1:] - off[:-1]
        start = torch.zeros_like(off)
        start[1:] = ((n + BLK - 1) // BLK * BLK).cumsum(0)
        p = torch.arange(P, device=v.device)
        e = (torch.searchsorted(start, p, right=True) - 1).clamp_max(n.numel() - 1)
        row = p - start[e]
        there = row < n[e]
        src = s["index"].long()[torch.where(there, off[e] + row, 0)]
        v = torch.where(there[:, None], v[src], 0.0)
    b = v.view(-1, BLK, v.shape[1])
    r, sc = _factors(b.abs().amax(1))
    codes = _to_codes(b * r[:, None, :]).view(P, -1).t().contiguous()
    if s["offsets"] is not None:
        sc = torch.where(torch.arange(P // BLK, device=v.device)[:, None] * BLK < start[-1], sc, 0.0)
    return codes, sc


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        y, _, _ = _norm_plain(s["x"], s["weight"], s["bias"], c["center"])
        if c["out"] == "codes":
            codes, scales = _rows_plain(y)
            return [_stands_for(codes), scales]
        return y.to(_DTYPE[c["out"]])
    if op == "norm_train":
        y, mean, rstd = _norm_plain(s["x"], s["weight"], s["bias"], c["center"])
        out = {"mean": mean, "rstd": rstd}
        if c["checkpoint"]:
            codes, scales = _rows_plain(y)
            kept, kept_scales = _rows_plain(s["x"])
            x = _values(kept, kept_scales)
            out.update(y=_stands_for(codes), y_scales=scales, x=_stands_for(kept),
                       x_scales=kept_scales)
        else:
            x = s["x"].float()
            out["y"] = y.bfloat16()
        dx, dweight, dbias = _norm_backward_plain(s["dy"], x, mean, rstd, s["weight"], c["center"])
        out.update(dx=dx.to(s["x"].dtype), dweight=dweight, dbias=dbias)
        return out
    if op in ("act", "act_train"):
        H = c["H"]
        u = s["u"].float()
        h, _ = _act_plain(u[:, :H], c["kind"])
        codes, scales = _rows_plain(h * u[:, H:] if c["gated"] else h)
        out = {"h": _stands_for(codes), "h_scales": scales}
        if op == "act":
            return out
        kept, kept_scales = _rows_plain(s["u"])
        u = _values(kept, kept_scales)
        h, d = _act_plain(u[:, :H], c["kind"])
        dh = s["dh"].float()
        du = torch.cat([dh * u[:, H:] * d, dh * h], 1) if c["gated"] else dh * d
        codes, scales = _rows_plain(du)
        out.update(u=_stands_for(kept), u_scales=kept_scales, du=du.bfloat16(),
                   du_codes=_stands_for(codes), du_scales=scales)
        return out
    if op == "cols":
        codes, scales = _cols_plain(s)
        return [_stands_for(codes), scales]
    codes, scales = s["codes"], s["scales"]
    if s["index"] is not None:
        codes, scales = codes[s["index"].long()], scales[:, s["index"].long()]
    return _values(codes, scales).to(_DTYPE[c["out"]])


# ---------------------------------------------------------------------------------------------
# the framework's operators
# ---------------------------------------------------------------------------------------------
def _run_own(s):
    import mx_microscaling_quantize_gb300 as mxq

    c = s["case"]
    op = c["op"]
    if op == "norm":
        if c["out"] == "codes":
            codes, scales = mxq.mx_layer_norm_b128(s["x"], s["weight"], s["bias"], eps=EPS,
                                                   center=c["center"])
            return [_stands_for(codes), scales]
        return mxq.mx_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, center=c["center"],
                                 out_dtype=_DTYPE[c["out"]])
    if op == "norm_train":
        x, x_scales = s["x"], None
        if c["checkpoint"]:
            codes, scales, mean, rstd, x, x_scales = mxq.mx_layer_norm_b128(
                s["x"], s["weight"], s["bias"], eps=EPS, center=c["center"], stats=True,
                checkpoint=True)
            out = {"y": _stands_for(codes), "y_scales": scales, "x": _stands_for(x),
                   "x_scales": x_scales}
        else:
            y, mean, rstd = mxq.mx_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS,
                                              center=c["center"], out_dtype=torch.bfloat16,
                                              stats=True)
            out = {"y": y}
        dx, dweight, dbias = mxq.mx_layer_norm_backward(
            s["dy"], x, mean, rstd, s["weight"], x_scales=x_scales, bias_grad=c["center"],
            out_dtype=s["x"].dtype)
        out.update(mean=mean, rstd=rstd, dx=dx, dweight=dweight, dbias=dbias)
        return out
    if op in ("act", "act_train"):
        kind = {"silu": mxq.SILU, "gelu": mxq.GELU, "gelu_tanh": mxq.GELU_TANH}[c["kind"]]
        if op == "act":
            codes, scales = mxq.mx_activation_b128(s["u"], kind, gated=c["gated"])
            return {"h": _stands_for(codes), "h_scales": scales}
        codes, scales, kept, kept_scales = mxq.mx_activation_b128(s["u"], kind, gated=c["gated"],
                                                                  checkpoint=True)
        du, du_codes, du_scales = mxq.mx_activation_backward(
            s["dh"], kept, kind, gated=c["gated"], u_scales=kept_scales, operand=True)
        return {"h": _stands_for(codes), "h_scales": scales, "u": _stands_for(kept),
                "u_scales": kept_scales, "du": du, "du_codes": _stands_for(du_codes),
                "du_scales": du_scales}
    if op == "cols":
        codes, scales = mxq.mx_requantize_b128_cols(s["codes"], s["scales"], s["index"],
                                                    s["offsets"], out_codes=s["out_codes"],
                                                    out_scales=s["out_scales"])
        return [_stands_for(codes), scales]
    return mxq.mx_dequantize_b128_rows(s["codes"], s["scales"], s["index"],
                                       out_dtype=_DTYPE[c["out"]])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def _e4m3_round(t):
    """Nearest E4M3 value, ties to even, of the (saturated) 64-bit values t."""
    t = t.clamp(-448.0, 448.0)
    _, e = torch.frexp(t)  # |t| in [2^(e-1), 2^e): 3 fraction bits, least exponent -6
    spacing = torch.tensor([2.0 ** i for i in range(-9, 6)], dtype=t.dtype, device=t.device)
    q = spacing[(e.long() + 5).clamp_min(0)]
    return torch.round(t / q) * q


def _blocks_exact(v, dim):
    """Grid values and scales [blocks, rows or columns] of blocks of 128 along dim. A block's factors
    and the scaled element are defined in 32 bits where v is, else taken in 64."""
    grids, scales = [], []
    for part in v.split(BLK, dim):
        a = part.abs().amax(dim, keepdim=True).clamp_min(2.0 ** -100)
        grids.append(_e4m3_round((part * (torch.full_like(a, 448.0) / a)).double()))
        scales.append((a / 448.0).double().flatten())
    return torch.cat(grids, dim), torch.stack(scales)


def _stored(v):
    """v after a round trip through a checkpoint: grid, scales and (in 32 bits, as defined) values."""
    grid, scales = _blocks_exact(v.float(), 1)
    per = scales.float().t().repeat_interleave(BLK, 1)[:, :v.shape[1]]
    return grid, scales, grid.float() * per


def _decoded(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float()
    return torch.cat([p * scales[j][:, None] for j, p in enumerate(v.split(BLK, 1))], 1)


def _act_exact(g, kind):
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if kind == "gelu":
        p = torch.special.ndtr(g)
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    d = 0.5 * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + g * d


def _exact_norm(s):
    c = s["case"]
    x, w = s["x"].double(), s["weight"].double()
    mean = x.mean(1, keepdim=True) if c["center"] else torch.zeros_like(x[:, :1])
    rstd = torch.rsqrt((x - mean).square().mean(1, keepdim=True) + EPS)
    y = (x - mean) * rstd * w
    if s["bias"] is not None:
        y = y + s["bias"].double()
    if c["op"] == "norm":
        return list(_blocks_exact(y, 1)) if c["out"] == "codes" else y
    out = {"mean": mean[:, 0] if c["center"] else None, "rstd": rstd[:, 0]}
    if c["checkpoint"]:
        out["y"], out["y_scales"] = _blocks_exact(y, 1)
        out["x"], out["x_scales"], x = _stored(s["x"])
        x = x.double()
    else:
        out["y"] = y
    xhat, dy = (x - mean) * rstd, s["dy"].double()
    g = dy * w
    dx = g - xhat * (g * xhat).mean(1, keepdim=True)
    if c["center"]:
        dx = dx - g.mean(1, keepdim=True)
    out.update(dx=dx * rstd, dweight=(dy * xhat).sum(0), dbias=dy.sum(0) if c["center"] else None)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_train"):
        return _exact_norm(s)
    if op in ("act", "act_train"):
        H, gated = case["H"], case["gated"]
        u = s["u"].double()
        h = _act_exact(u[:, :H], case["kind"])[0]
        out = {}
        out["h"], out["h_scales"] = _blocks_exact(h * u[:, H:] if gated else h, 1)
        if op == "act":
            return out
        out["u"], out["u_scales"], u = _stored(s["u"])
        u = u.double()
        h, d = _act_exact(u[:, :H], case["kind"])
        dh = s["dh"].double()
        out["du"] = torch.cat([dh * u[:, H:] * d, dh * h], 1) if gated else dh * d
        out["du_codes"], out["du_scales"] = _blocks_exact(out["du"], 1)
        return out
    v = _decoded(s["codes"], s["scales"])
    if op == "cols":
        K, P = case["K"], s["out_codes"].shape[1]
        grid = torch.zeros(K, P, dtype=torch.float64, device=v.device)
        scales = torch.zeros(P // BLK, K, dtype=torch.float64, device=v.device)
        at = [0, v.shape[0]] if s["offsets"] is None else s["offsets"].tolist()
        rows = v if s["index"] is None else v[s["index"].long()]
        p = 0
        for lo, hi in zip(at[:-1], at[1:]):
            if hi > lo:
                g, sc = _blocks_exact(rows[lo:hi], 0)
                grid[:, p:p + hi - lo] = g.t()
                scales[p // BLK:p // BLK + sc.shape[0]] = sc
                p += sc.shape[0] * BLK
        return [grid, scales]
    v = v.double() if s["index"] is None else v[s["index"].long()].double()
    return v
