"""What is measured of the expert-layer operators: routing, 8-bit quantisation with a scale per
block of 128, the product of such operands (dense and by expert) and the combination of the
experts' outputs.

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


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of a serving step picking 8 of 128 experts
        dict(name="route_one_token", op="route", T=1, E=128, k=8, score="softmax", bias=False,
             groups=1, top=1, renorm=True, dtype="bf16", train=False),
        # a long prompt, 256 experts in 8 groups of which 4 stay, balance bias, sigmoid scores
        dict(name="route_grouped_prompt", op="route", T=16384, E=256, k=8, score="sigmoid",
             bias=True, groups=8, top=4, renorm=True, dtype="fp32", train=False),
        # a training step's router: softmax weights as they are, gradient to every logit
        dict(name="route_train", op="route", T=4097, E=64, k=6, score="softmax", bias=False,
             groups=1, top=1, renorm=False, dtype="bf16", train=True),
        # the smallest activation of the library's workloads
        dict(name="quantize_rows_small", op="quantize", kind="rows", M=128, K=4096, R=0),
        # the weight-gradient operand of a large activation: transposed, scales along the tokens
        dict(name="quantize_cols_large", op="quantize", kind="cols", M=8192, K=8192, R=0),
        # one token through a large layer
        dict(name="linear_decode", op="linear", M=1, N=8192, K=8192, train=False),
        # a prompt of 8192 tokens through the same layer
        dict(name="linear_prompt", op="linear", M=8192, N=8192, K=8192, train=False),
        # a training step of a layer on a ragged batch: quantise, product, both gradients
        dict(name="linear_train_ragged", op="linear", M=4001, N=2048, K=8192, train=True),
        # 16 tokens of a serving step through 8 of 128 experts each
        dict(name="experts_decode", op="experts", T=16, k=8, E=128, K=2048, N=1024, skew=0.0,
             train=False),
        # a training step: 16384 expert rows over 128 unevenly loaded experts
        dict(name="experts_train", op="experts", T=4096, k=4, E=128, K=2048, N=1024, skew=1.1,
             train=True),
        # the outputs of a serving step's experts joined
        dict(name="combine_decode", op="combine", T=16, k=8, N=2048, train=False),
        # the same for a training batch, with its gradients
        dict(name="combine_train", op="combine", T=16384, k=8, N=2048, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "quantize", "linear", "experts", "combine"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * rng.randint(2, 512 // groups)
        top = rng.randint(1, groups)
        k = rng.randint(1, min(16, E // groups * top))
        score = rng.choice(("softmax", "sigmoid"))
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, score=score,
                    bias=score == "sigmoid" and rng.random() < 0.5, groups=groups, top=top,
                    renorm=rng.random() < 0.5, dtype=rng.choice(("bf16", "fp32")),
                    train=rng.random() < 0.4)
    if op == "quantize":
        kind = rng.choice(("rows", "gather", "blocks", "cols"))
        M, K = _log(rng, 1, 8192), 32 * _log(rng, 1, 256)
        return dict(op=op, kind=kind, M=M, K=K, R=_log(rng, 1, 8192) if kind == "gather" else 0)
    if op == "linear":
        train = rng.random() < 0.4
        if train:
            return dict(op=op, M=_log(rng, 16, 4096), N=32 * _log(rng, 4, 128),
                        K=32 * _log(rng, 4, 256), train=True)
        return dict(op=op, M=_log(rng, 1, 8192), N=8 * _log(rng, 16, 1024),
                    K=32 * _log(rng, 4, 256), train=False)
    if op == "experts":
        E = _log(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        return dict(op=op, T=_log(rng, 1, 16384 // k), k=k, E=E, K=32 * _log(rng, 8, 64),
                    N=32 * _log(rng, 8, 32), skew=rng.choice((0.0, 1.1)),
                    train=rng.random() < 0.4)
    return dict(op=op, T=_log(rng, 1, 16384), k=rng.randint(1, 8), N=8 * _log(rng, 16, 256),
                train=rng.random() < 0.5)


def _touched(case):
    """Expected number of experts that at least one token chooses."""
    p = [(e + 1) ** -case["skew"] for e in range(case["E"])]
    s = sum(p)
    return sum(1 - (1 - min(1.0, case["k"] * q / s)) ** case["T"] for q in p)


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        el = 2 if case["dtype"] == "bf16" else 4
        b = T * E * el + T * k * 16 + 8 * (E + 1)
        if case["train"]:
            b += T * E * el + T * k * 4
        return {"bytes": b, "flops": T * E * 4}
    if op == "quantize":
        rows = case["R"] or case["M"]
        n = rows * case["K"]
        sc = 4 * n / BLK if case["kind"] != "blocks" else 4 * n / (BLK * BLK)
        if case["kind"] == "blocks":
            return {"bytes": 2 * n + 2 * (n + sc), "flops": 2 * n}
        return {"bytes": 2 * min(rows, case["M"]) * case["K"] + n + sc, "flops": 2 * n}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        if case["train"]:  # bf16 x, w, dy in; bf16 y, dx and fp32 dw out
            return {"bytes": 4 * (M * K + M * N) + 6 * N * K, "flops": 6 * M * N * K}
        return {"bytes": M * K + N * K + 4 * M * K / BLK + 2 * M * N, "flops": 2 * M * N * K}
    if op == "experts":
        T, N, K, E = case["T"], case["N"], case["K"], case["E"]
        R, used = T * case["k"], _touched(case)
        b = 2 * T * K + used * N * K + 2 * R * N
        if case["train"]:
            return {"bytes": b + 2 * R * N + used * N * K + 2 * T * K + 4 * E * N * K,
                    "flops": 6 * R * N * K}
        return {"bytes": b, "flops": 2 * R * N * K}
    T, k, N = case["T"], case["k"], case["N"]
    b = 2 * T * k * N + 2 * T * N + 8 * T * k
    if case["train"]:
        b += 2 * T * N + 2 * T * k * N + 4 * T * k
    return {"bytes": b, "flops": 2 * T * k * N * (3 if case["train"] else 1)}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _activations(M, K, gen):
    """Normal activations with a few loud channels, bf16."""
    x = torch.randn(M, K, generator=gen, device=DEV)
    loud = torch.rand(K, generator=gen, device=DEV) < 0.005
    return (x * torch.where(loud, 20.0, 1.0)).bfloat16()


def _choices(T, k, E, skew, gen):
    """k distinct experts for each token, by popularity rank^-skew under a random order."""
    logp = -skew * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    logp = logp[torch.randperm(E, generator=gen, device=DEV)]
    u = torch.rand(T, E, generator=gen, device=DEV).clamp_min(1e-12)
    return torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices.int().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "route":
        T, E = case["T"], case["E"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["logits"] = (torch.randn(T, E, generator=gen, device=DEV) * 1.5).to(dt)
        s["bias"] = (torch.randn(E, generator=gen, device=DEV) * 0.05) if case["bias"] else None
        if case["train"]:
            s["grad"] = torch.randn(T, case["k"], generator=gen, device=DEV)
        return s
    if op == "quantize":
        s["x"] = _activations(case["M"], case["K"], gen)
        s["index"] = None
        if case["kind"] == "gather":
            s["index"] = torch.randint(0, case["M"], (case["R"],), generator=gen, device=DEV,
                                       dtype=torch.int32)
        return s
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        x = _activations(M, K, gen)
        w = (torch.randn(N, K, generator=gen, device=DEV) * 0.02).bfloat16()
        if case["train"]:
            s["x"], s["w"] = x, w
            s["dy"] = (torch.randn(M, N, generator=gen, device=DEV) * 1e-3).bfloat16()
        else:
            s["a"], s["b"] = _rows_plain(x), _blocks_plain(w)
        return s
    if op == "experts":
        T, k, E, N, K = case["T"], case["k"], case["E"], case["N"], case["K"]
        s["x"] = _activations(T, K, gen)
        w = (torch.randn(E, N, K, generator=gen, device=DEV) * 0.02).bfloat16()
        s["plan"] = _plan_plain(_choices(T, k, E, case["skew"], gen), E)
        s["w"] = _blocks_plain(w)
        if case["train"]:
            s["wt"] = tuple(t.transpose(-1, -2).contiguous() for t in s["w"])
            s["dy"] = (torch.randn(T * k, N, generator=gen, device=DEV) * 1e-3).bfloat16()
        return s
    T, k, N = case["T"], case["k"], case["N"]
    s["y"] = torch.randn(T * k, N, generator=gen, device=DEV).bfloat16()
    s["slots"] = torch.randperm(T * k, generator=gen, device=DEV).int().view(T, k)
    w = torch.rand(T, k, generator=gen, device=DEV) + 0.05
    s["weights"] = w / w.sum(1, keepdim=True)
    if case["train"]:
        s["dout"] = (torch.randn(T, N, generator=gen, device=DEV) * 1e-2).bfloat16()
    return s


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _to_codes(t):
    return t.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _factors(amax):
    a = amax.clamp_min(AMAX_FLOOR)
    return torch.full_like(a, E4M3_MAX) / a, a / E4M3_MAX


def _pad_to(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[-1], 0, rows - x.shape[-2]))


def _up(n):
    return -(-n // BLK) * BLK


def _rows_plain(x, index=None):
    """1 x 128 blocks: codes [R, K] as bytes, scales [K / 128, R]."""
    v = (x if index is None else x[index.long()]).float()
    R, K = v.shape
    b = _pad_to(v, R, _up(K)).view(R, -1, BLK)
    r, s = _factors(b.abs().amax(2))
    codes = _to_codes(b * r[:, :, None]).view(torch.uint8).view(R, -1)[:, :K]
    return codes.contiguous(), s.t().contiguous()


def _blocks_plain(w):
    """128 x 128 blocks: codes as w, scales [.., N / 128, K / 128]."""
    N, K = w.shape[-2:]
    b = _pad_to(w.float(), _up(N), _up(K)).view(-1, _up(N) // BLK, BLK, _up(K) // BLK, BLK)
    r, s = _factors(b.abs().amax((2, 4)))
    codes = _to_codes(b * r[:, :, None, :, None]).view(torch.uint8)
    codes = codes.view(*w.shape[:-2], _up(N), _up(K))[..., :N, :K].contiguous()
    return codes, s.view(*w.shape[:-2], _up(N) // BLK, _up(K) // BLK)


def _cols_plain(x):
    """128 x 1 blocks, transposed: codes [K, M'] as bytes, scales [M' / 128, K] (M' = M padded)."""
    M, K = x.shape
    b = _pad_to(x.float(), _up(M), K).view(-1, BLK, K)
    r, s = _factors(b.abs().amax(1))
    codes = _to_codes(b * r[:, None, :]).view(torch.uint8).view(-1, K)
    return codes.t().contiguous(), s


def _values(codes, scales):
    """Rows-form operand as its 32-bit values."""
    v = codes.view(torch.float8_e4m3fn).float()
    return v * scales.t().repeat_interleave(BLK, 1)[:, :v.shape[1]]


def _block_values(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float()
    s = scales.repeat_interleave(BLK, -1).repeat_interleave(BLK, -2)
    return v * s[..., :v.shape[-2], :v.shape[-1]]


def _plan_plain(experts, E):
    T, k = experts.shape
    flat = experts.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    counts = torch.bincount(key, minlength=E + 1)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    offsets[1:] = counts[:E].cumsum(0)
    order = torch.sort(key, stable=True).indices
    n = torch.arange(T * k, device=flat.device)
    made = n < offsets[E]
    tokens = torch.where(made, order // k, -1).int()
    slots = torch.empty_like(n)
    slots[order] = torch.where(made, n, -1)
    return offsets, tokens, slots.int().view(T, k)


def _scores_plain(logits, score):
    """-> unnormalised scores and what they are divided by."""
    l = logits.float()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l)), None
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e, e.sum(1, keepdim=True)


def _route_plain(logits, k, score, bias, groups, top, renorm):
    T, E = logits.shape
    s, total = _scores_plain(logits, score)
    choice = s if bias is None else s + bias
    choice = torch.where(torch.isneginf(logits), -math.inf, choice)
    if groups > 1:
        best = choice.view(T, groups, -1).sort(dim=2, descending=True).values[:, :, :2]
        second = torch.where(torch.isneginf(best[:, :, 1]), 0.0, best[:, :, 1])
        kept = (best[:, :, 0] + second).sort(dim=1, descending=True, stable=True).indices[:, :top]
        keep = torch.zeros(T, groups, dtype=torch.bool, device=logits.device)
        keep.scatter_(1, kept, True)
        choice = torch.where(keep.repeat_interleave(E // groups, 1), choice, -math.inf)
    value, index = choice.sort(dim=1, descending=True, stable=True)
    index = index[:, :k]
    made = ~torch.isneginf(value[:, :k])
    w = s.gather(1, index)
    if total is not None:
        w = w / total
    w = torch.where(made, w, 0.0)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    return torch.where(made, index, -1).int(), w


def _route_backward_plain(grad, logits, experts, score, renorm):
    s, total = _scores_plain(logits, score)
    if total is not None:
        s = s / total
    index = experts.long().clamp_min(0)
    made = experts >= 0
    p = torch.where(made, s.gather(1, index), 0.0)
    dp = torch.where(made, grad, 0.0)
    if renorm:
        P = p.sum(1, keepdim=True)
        dp = torch.where(made, (dp - (dp * p).sum(1, keepdim=True) / P) / P, 0.0)
    ds = torch.zeros_like(s).scatter_add_(1, index, dp)
    if score == "sigmoid":
        d = ds * s * (1.0 - s)
    else:
        d = s * (ds - (ds * s).sum(1, keepdim=True))
    return d.to(logits.dtype)


def _experts_plain(a, w, offsets):
    """Rows [offsets[e], offsets[e + 1]) of the values a times expert e's values transposed."""
    at = offsets.tolist()
    out = torch.empty(a.shape[0], w.shape[1], device=a.device)
    for e in range(w.shape[0]):
        if at[e + 1] > at[e]:
            torch.mm(a[at[e]:at[e + 1]], w[e].t(), out=out[at[e]:at[e + 1]])
    return out.bfloat16()


def _experts_wgrad_plain(dy, x, offsets, E):
    """dw[e] = dy_e^T x_e, each expert's operands quantised along its own rows (padded to 128)."""
    at = offsets.tolist()
    dw = torch.zeros(E, dy.shape[1], x.shape[1], device=x.device)
    for e in range(E):
        if at[e + 1] > at[e]:
            u = _values(*_cols_plain(dy[at[e]:at[e + 1]]))
            v = _values(*_cols_plain(x[at[e]:at[e + 1]]))
            torch.mm(u, v.t(), out=dw[e])
    return dw


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        experts, weights = _route_plain(s["logits"], c["k"], c["score"], s["bias"], c["groups"],
                                        c["top"], c["renorm"])
        out = [experts, weights, *_plan_plain(experts, c["E"])]
        if c["train"]:
            out.append(_route_backward_plain(s["grad"], s["logits"], experts, c["score"],
                                             c["renorm"]))
        return out
    if op == "quantize":
        if c["kind"] == "cols":
            codes, scales = _cols_plain(s["x"])
        elif c["kind"] == "blocks":
            codes, scales = _blocks_plain(s["x"])
            return [codes.view(torch.float8_e4m3fn), scales,
                    codes.t().contiguous().view(torch.float8_e4m3fn), scales.t().contiguous()]
        else:
            codes, scales = _rows_plain(s["x"], s["index"])
        return [codes.view(torch.float8_e4m3fn), scales]
    if op == "linear":
        if not c["train"]:
            return (_values(*s["a"]) @ _block_values(*s["b"]).t()).bfloat16()
        w = _block_values(*_blocks_plain(s["w"]))
        y = (_values(*_rows_plain(s["x"])) @ w.t()).bfloat16()
        dx = (_values(*_rows_plain(s["dy"])) @ w).bfloat16()
        dw = _values(*_cols_plain(s["dy"])) @ _values(*_cols_plain(s["x"])).t()
        return {"y": y, "dx": dx, "dw": dw}
    if op == "experts":
        offsets, tokens, slots = s["plan"]
        w = _block_values(*s["w"])
        y = _experts_plain(_values(*_rows_plain(s["x"], tokens)), w, offsets)
        if not c["train"]:
            return y
        d = _experts_plain(_values(*_rows_plain(s["dy"])), w.transpose(1, 2), offsets)
        dx = d[slots.long()].float().sum(1).bfloat16()
        dw = _experts_wgrad_plain(s["dy"], s["x"][tokens.long()], offsets, c["E"])
        return {"y": y, "dx": dx, "dw": dw}
    rows = s["y"][s["slots"].long()].float()
    out = (rows * s["weights"][:, :, None]).sum(1).bfloat16()
    if not c["train"]:
        return out
    dout = s["dout"].float()
    dy = torch.empty_like(s["y"])
    dy[s["slots"].long()] = (s["weights"][:, :, None] * dout[:, None, :]).bfloat16()
    dweights = (rows * dout[:, None, :]).sum(2)
    return {"out": out, "dy": dy, "dweights": dweights}


# ---------------------------------------------------------------------------------------------
# the framework's operators
# ---------------------------------------------------------------------------------------------
def _run_own(s):
    import mx_microscaling_quantize_gb300 as mxq

    c = s["case"]
    op = c["op"]
    if op == "route":
        score = mxq.SOFTMAX if c["score"] == "softmax" else mxq.SIGMOID
        experts, weights = mxq.mx_route(s["logits"], c["k"], score, s["bias"], groups=c["groups"],
                                        top_groups=c["top"], renormalize=c["renorm"])
        out = [experts, weights, *mxq.mx_route_plan(experts, c["E"])]
        if c["train"]:
            out.append(mxq.mx_route_backward(s["grad"], s["logits"], experts, score,
                                             renormalize=c["renorm"]))
        return out
    if op == "quantize":
        if c["kind"] == "blocks":
            codes, scales, tcodes, tscales = mxq.mx_quantize_b128_blocks(s["x"], transpose=True)
            return [codes.view(torch.float8_e4m3fn), scales, tcodes.view(torch.float8_e4m3fn),
                    tscales]
        if c["kind"] == "cols":
            codes, scales = mxq.mx_quantize_b128_cols(s["x"])
        else:
            codes, scales = mxq.mx_quantize_b128_rows(s["x"], s["index"])
        return [codes.view(torch.float8_e4m3fn), scales]
    if op == "linear":
        if not c["train"]:
            return mxq.mx_gemm_b128(*s["a"], *s["b"])
        wq, ws, wtq, wts = mxq.mx_quantize_b128_blocks(s["w"], transpose=True)
        y = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_rows(s["x"]), wq, ws)
        dx = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_rows(s["dy"]), wtq, wts)
        dw = mxq.mx_gemm_b128(*mxq.mx_quantize_b128_cols(s["dy"]),
                              *mxq.mx_quantize_b128_cols(s["x"]), mxq.B128_ROWS,
                              out_dtype=torch.float32)
        return {"y": y, "dx": dx, "dw": dw}
    if op == "experts":
        offsets, tokens, slots = s["plan"]
        y = mxq.mx_gemm_b128_grouped(*mxq.mx_quantize_b128_rows(s["x"], tokens), *s["w"], offsets)
        if not c["train"]:
            return y
        d = mxq.mx_gemm_b128_grouped(*mxq.mx_quantize_b128_rows(s["dy"]), *s["wt"], offsets)
        dx = mxq.mx_combine(d, slots)
        dw = mxq.mx_gemm_b128_grouped_wgrad(
            *mxq.mx_quantize_b128_cols(s["dy"], row_offsets=offsets),
            *mxq.mx_quantize_b128_cols(s["x"], tokens, offsets), offsets,
            out_dtype=torch.float32)
        return {"y": y, "dx": dx, "dw": dw}
    out = mxq.mx_combine(s["y"], s["slots"], s["weights"])
    if not c["train"]:
        return out
    dy, dweights = mxq.mx_combine_backward(s["dout"], s["y"], s["slots"], s["weights"])
    return {"out": out, "dy": dy, "dweights": dweights}


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


def _quantized(x, dim):
    """Values that 1 x 128 (dim 1) or 128 x 1 (dim 0) blocks of x [M, K] stand for, in 64 bits.
    The two factors are defined in 32 bits: 448 / a and a / 448, and so is the scaled element."""
    return torch.cat([_quantized_block(part, dim) for part in x.split(BLK, dim)], dim)


def _quantized_block(x, dim):
    v = x.to(torch.float32)
    a = torch.maximum(v.abs().max(dim, keepdim=True).values,
                      torch.full((), 2.0 ** -100, device=v.device))
    grid = _e4m3_round((v * torch.div(torch.full_like(a, 448.0), a)).double())
    return grid * (a / 448.0).double()


def _quantized_square(w):
    out = torch.empty(w.shape, dtype=torch.float64, device=w.device)
    for i in range(0, w.shape[0], BLK):
        for j in range(0, w.shape[1], BLK):
            part = w[i:i + BLK, j:j + BLK]
            out[i:i + BLK, j:j + BLK] = _quantized_block(part.reshape(1, -1), 1).view(part.shape)
    return out


def _decode(codes, scales, square):
    """64-bit values of codes [rows, K] under scales [K / 128, rows] or [rows / 128, K / 128]."""
    v = codes.view(torch.float8_e4m3fn).double()
    for j in range(0, v.shape[1], BLK):
        if square:
            col = scales[:, j // BLK].double()
            v[:, j:j + BLK] *= col[torch.arange(v.shape[0], device=v.device) // BLK][:, None]
        else:
            v[:, j:j + BLK] *= scales[j // BLK].double()[:, None]
    return v


def _exact_route(s):
    c = s["case"]
    l = s["logits"].double()
    T, E = l.shape
    if c["score"] == "sigmoid":
        p = torch.sigmoid(l)
    else:
        p = torch.softmax(l, 1)
    choice = p if s["bias"] is None else p + s["bias"].double()
    if c["groups"] > 1:
        g = torch.topk(choice.view(T, c["groups"], -1), 2, 2).values.sum(2)
        bar = torch.topk(g, c["top"], 1).values[:, -1:]
        choice = choice.masked_fill((g < bar).repeat_interleave(E // c["groups"], 1), -math.inf)
    index = choice.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = p.gather(1, index)
    P = w.sum(1, keepdim=True)
    out = [None, w / P if c["renorm"] else w, None, None, None]
    if c["train"]:
        g = s["grad"].double()
        if c["renorm"]:
            g = (g - (g * w / P).sum(1, keepdim=True)) / P
        full = torch.zeros_like(p).scatter_(1, index, g)
        if c["score"] == "sigmoid":
            out.append(full * p * (1 - p))
        else:
            out.append(p * (full - (full * p).sum(1, keepdim=True)))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "quantize":
        x, kind = s["x"], case["kind"]
        v = x if kind != "gather" else x[s["index"].long()]
        v = v.t() if kind == "cols" else v
        R, K = v.shape
        Kp = -(-K // BLK) * BLK
        if kind == "blocks":
            full = torch.zeros(-(-R // BLK) * BLK, Kp, device=v.device)
            full[:R, :K] = v.float().abs()
            a = full.view(-1, BLK, Kp // BLK, BLK).amax((1, 3)).clamp_min(2.0 ** -100)
            per = a.repeat_interleave(BLK, 0).repeat_interleave(BLK, 1)[:R, :K]
        else:
            full = torch.zeros(R, Kp, device=v.device)
            full[:, :K] = v.float().abs()
            a = full.view(R, -1, BLK).amax(2).clamp_min(2.0 ** -100)
            per = a.repeat_interleave(BLK, 1)[:, :K]
        grid = _e4m3_round((v.float() * torch.div(torch.full_like(per, 448.0), per)).double())
        scales = a.double() / 448.0
        if kind == "blocks":
            return [grid, scales, grid.t().contiguous(), scales.t().contiguous()]
        if kind == "cols":
            grid = torch.nn.functional.pad(grid, (0, Kp - K))
        return [grid, scales.t().contiguous()]
    if op == "linear":
        if not case["train"]:
            return _decode(*s["a"], False) @ _decode(*s["b"], True).t()
        w = _quantized_square(s["w"])
        return {"y": _quantized(s["x"], 1) @ w.t(), "dx": _quantized(s["dy"], 1) @ w,
                "dw": _quantized(s["dy"], 0).t() @ _quantized(s["x"], 0)}
    if op == "experts":
        offsets, tokens, _ = s["plan"]
        at = offsets.tolist()
        x = s["x"][tokens.long()]
        rows = _quantized(x, 1)
        y = torch.empty(x.shape[0], case["N"], dtype=torch.float64, device=x.device)
        train = case["train"]
        if train:
            drows = _quantized(s["dy"], 1)
            dx = torch.zeros(case["T"], case["K"], dtype=torch.float64, device=x.device)
            dw = torch.zeros(case["E"], case["N"], case["K"], dtype=torch.float64,
                             device=x.device)
        for e in range(case["E"]):
            lo, hi = at[e], at[e + 1]
            if lo == hi:
                continue
            w = _decode(s["w"][0][e], s["w"][1][e], True)
            y[lo:hi] = rows[lo:hi] @ w.t()
            if train:
                dx.index_add_(0, tokens[lo:hi].long(), drows[lo:hi] @ w)
                dw[e] = _quantized(s["dy"][lo:hi], 0).t() @ _quantized(x[lo:hi], 0)
        return {"y": y, "dx": dx, "dw": dw} if train else y
    T, k, N = case["T"], case["k"], case["N"]
    out = torch.zeros(T, N, dtype=torch.float64, device=DEV)
    for j in range(k):
        out += s["y"][s["slots"][:, j].long()].double() * s["weights"][:, j:j + 1].double()
    if not case["train"]:
        return out
    dy = torch.empty(T * k, N, dtype=torch.float64, device=DEV)
    dweights = torch.empty(T, k, dtype=torch.float64, device=DEV)
    for j in range(k):
        at = s["slots"][:, j].long()
        dy[at] = s["dout"].double() * s["weights"][:, j:j + 1].double()
        dweights[:, j] = (s["dout"].double() * s["y"][at].double()).sum(1)
    return {"out": out, "dy": dy, "dweights": dweights}
