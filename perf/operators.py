"""Cases that measure the operators around the MoE layer on one GPU.

  norm      residual addition + root-mean-square norm, written as bf16 rows
            (what the router reads) and / or as e4m3 codes with one UE8M0
            scale byte per 32 values (what low-bit experts read)
  linear    out = act(x w^T + bias) + residual with bf16 operands: the shared
            expert and the gate's logits beside the routed experts
  balance   expert-load balance loss, per-expert counts and the gradient of
            the gate's logits

`own = False` runs every operator in its plain form (elementary torch
operations in 32 bits, rounded once at the end); `own = True` runs the
library's entry points on the same inputs.  `exact` states the definitions in
64 bits, apart from both.
"""
import math

import torch

own = False

_moe = None


def _lib():
    global _moe
    if _moe is None:
        from router_experts_gb300 import moe
        _moe = moe
    return _moe


# ---- cases ----------------------------------------------------------------------

def listed():
    return [
        # one decoded token of the DeepSeek-V3 layer: pure latency
        {"name": "norm decode 1x7168", "op": "norm", "T": 1, "H": 7168, "x": "bf16",
         "res": "bf16", "w": "bf16", "y": True, "e4m3": False},
        # a decode batch in front of the low-bit layer: router rows and expert codes
        {"name": "norm batch 64x4096 e4m3", "op": "norm", "T": 64, "H": 4096, "x": "bf16",
         "res": "bf16", "w": "bf16", "y": True, "e4m3": True},
        # odd row width and a ragged token count, no 16-byte vectors anywhere
        {"name": "norm odd 1021x2045", "op": "norm", "T": 1021, "H": 2045, "x": "bf16",
         "res": "f32", "w": "f32", "y": True, "e4m3": False},
        # prefill with every output: HBM-bound
        {"name": "norm prefill 4096x7168 e4m3", "op": "norm", "T": 4096, "H": 7168, "x": "bf16",
         "res": "bf16", "w": "bf16", "y": True, "e4m3": True},
        # shared expert of one decoded token, gate and up rows in one matrix:
        # a 58.7 MB weight stream
        {"name": "linear decode swiglu 1x7168x2048", "op": "linear", "T": 1, "K": 7168, "N": 2048,
         "act": "swiglu", "bias": False, "res": "none", "out": "bf16"},
        # its down projection for a decode batch, added to the routed experts' output
        {"name": "linear batch residual 64x2048x7168", "op": "linear", "T": 64, "K": 2048,
         "N": 7168, "act": "none", "bias": False, "res": "bf16", "out": "bf16"},
        # logits of a 256-expert gate kept in 32 bits for the loss below
        {"name": "linear logits 512x7168x256 f32", "op": "linear", "T": 512, "K": 7168, "N": 256,
         "act": "none", "bias": False, "res": "none", "out": "f32"},
        # ragged in every direction, bias and activation
        {"name": "linear ragged 1023x4088x2001 gelu", "op": "linear", "T": 1023, "K": 4088,
         "N": 2001, "act": "gelu", "bias": True, "res": "bf16", "out": "bf16"},
        # shared expert of a prefill: tensor-bound
        {"name": "linear prefill swiglu 4096x7168x2048", "op": "linear", "T": 4096, "K": 7168,
         "N": 2048, "act": "swiglu", "bias": False, "res": "none", "out": "bf16"},
        # load statistics and loss of a decode batch: latency
        {"name": "balance 64x128", "op": "balance", "T": 64, "E": 128, "k": 8,
         "scoring": "softmax", "B": 1, "masked": False, "dt": "f32", "mode": "fused"},
        # one training step's tokens in ragged, padded sequences; the loss is
        # one term of several, so its gradient arrives from outside
        {"name": "balance 8192x256 ragged", "op": "balance", "T": 8192, "E": 256, "k": 8,
         "scoring": "sigmoid", "B": 7, "masked": True, "dt": "f32", "mode": "separate"},
        # a large training batch, loss and gradient in one call
        {"name": "balance 65536x256", "op": "balance", "T": 65536, "E": 256, "k": 8,
         "scoring": "sigmoid", "B": 16, "masked": False, "dt": "f32", "mode": "fused"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "balance"])
    if op == "norm":
        e4m3 = rng.random() < 0.5
        H = 32 * _log(rng, 2, 256) if e4m3 else _log(rng, 33, 8192)
        if not e4m3 and rng.random() < 0.5:
            H = (H + 7) // 8 * 8
        T = _log(rng, 1, min(16384, 4096 * 7168 // H))
        return {"op": op, "T": T, "H": H, "x": rng.choice(["bf16", "bf16", "f32"]),
                "res": rng.choice(["bf16", "bf16", "f32", "none"]),
                "w": rng.choice(["bf16", "f32"]), "y": not e4m3 or rng.random() < 0.6,
                "e4m3": e4m3}
    if op == "linear":
        K = 8 * _log(rng, 8, 1024)
        N = _log(rng, 17, 8192)
        if rng.random() < 0.6:
            N = (N + 31) // 32 * 32
        act = rng.choice(["none", "silu", "gelu", "swiglu"])
        rows = 2 * N if act == "swiglu" else N
        T = _log(rng, 1, max(1, min(8192, 4096 * 7168 * 4096 // (K * rows))))
        return {"op": op, "T": T, "K": K, "N": N, "act": act, "bias": rng.random() < 0.5,
                "res": rng.choice(["none", "bf16", "f32"]),
                "out": rng.choice(["bf16", "bf16", "f32"])}
    E = rng.choice([rng.randint(2, 64), rng.randint(65, 512), 128, 256, 288])
    k = rng.randint(1, min(16, E))
    T = _log(rng, 1, 65536 * 256 // max(E, 256))
    return {"op": op, "T": T, "E": E, "k": k,
            "scoring": rng.choice(["softmax", "sigmoid", "sqrt_softplus"]),
            "B": rng.randint(1, min(T, 16)), "masked": rng.random() < 0.5,
            "dt": rng.choice(["f32", "f32", "bf16"]),
            "mode": rng.choice(["fused", "separate", "forward"])}


# ---- inputs ---------------------------------------------------------------------

EPS = 1e-6
COEF = 1e-3
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(shape[0], -1)
    step = max(1, (1 << 26) // flat.shape[1])
    for r in range(0, shape[0], step):
        n = min(step, shape[0] - r)
        flat[r:r + n] = torch.randn((n, flat.shape[1]), generator=g, device="cuda") * std
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        # a residual stream: a few channels carry most of the energy
        gain = 1 + 15 * (torch.rand(H, generator=g, device="cuda") < 0.01).float()
        s["x"] = (torch.randn((T, H), generator=g, device="cuda") * 0.5).to(_DT[case["x"]])
        s["residual"] = None
        if case["res"] != "none":
            r = torch.randn((T, H), generator=g, device="cuda")
            s["residual"] = r.mul_(gain).to(_DT[case["res"]])
        s["weight"] = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(_DT[case["w"]])
        # the buffers a serving loop keeps for its outputs
        s["out"] = (torch.empty_like(s["residual"]) if case["res"] != "none" else None,
                    torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
                    if case["y"] else None,
                    torch.empty((T, H), dtype=torch.uint8, device="cuda")
                    if case["e4m3"] else None,
                    torch.empty((T, H // 32), dtype=torch.uint8, device="cuda")
                    if case["e4m3"] else None)
    elif case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        rows = 2 * N if case["act"] == "swiglu" else N
        s["x"] = _normal(g, T, K)
        s["w"] = _normal(g, rows, K, std=0.02)
        s["bias"] = torch.randn(rows, generator=g, device="cuda") if case["bias"] else None
        s["residual"] = (None if case["res"] == "none"
                         else _normal(g, T, N, dtype=_DT[case["res"]]))
        s["out"] = torch.empty((T, N), dtype=_DT[case["out"]], device="cuda")
    else:
        T, E, k, B = case["T"], case["E"], case["k"], case["B"]
        # popular and unpopular experts, as a router meets them before it is balanced
        offset = torch.randn(E, generator=g, device="cuda") * 0.5
        logits = (torch.randn((T, E), generator=g, device="cuda") + offset).to(_DT[case["dt"]])
        s["logits"] = logits
        s["topk_ids"] = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
        s["mask"] = None
        if case["masked"]:
            s["mask"] = torch.rand(T, generator=g, device="cuda") < 0.9
        s["seq_starts"] = None
        if B > 1:
            cuts = torch.randperm(T - 1, generator=g, device="cuda")[:B - 1] + 1
            s["seq_starts"] = torch.cat([cuts.new_zeros(1), cuts.sort().values,
                                         cuts.new_full((1,), T)]).to(torch.int32)
        s["dloss"] = torch.rand(1, generator=g, device="cuda") + 0.5
        s["out"] = (torch.empty(1, device="cuda"),
                    torch.empty((B, E), dtype=torch.int32, device="cuda"),
                    torch.empty(B, dtype=torch.int32, device="cuda"),
                    torch.empty_like(logits) if case["mode"] != "forward" else None)
    return s


# ---- one pass -------------------------------------------------------------------

def run(state):
    c = state["case"]
    if c["op"] == "norm":
        return _norm_own(state, c) if own else _norm_plain(state, c)
    if c["op"] == "linear":
        return _linear_own(state, c) if own else _linear_plain(state, c)
    return _balance_own(state, c) if own else _balance_plain(state, c)


def _norm_result(c, res, y, codes, scales):
    # codes and scale bytes as the numbers that they stand for
    out = {}
    if res is not None:
        out["residual"] = res
    if c["y"]:
        out["y"] = y
    if c["e4m3"]:
        out["codes"] = codes.view(torch.float8_e4m3fn)
        out["scales"] = scales.view(torch.float8_e8m0fnu)
    return out


def _norm_own(s, c):
    res, y, codes, scales = _lib().add_rms_norm(s["x"], s["weight"], s["residual"], EPS,
                                                y=c["y"], e4m3=c["e4m3"], out=s["out"])
    return _norm_result(c, res, y, codes, scales)


def _norm_plain(s, c):
    h = s["x"].float()
    res = None
    if s["residual"] is not None:
        h = h + s["residual"].float()
        res = h.to(s["residual"].dtype)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    codes = scales = None
    if c["e4m3"]:
        T, H = y.shape
        groups = y.view(T, H // 32, 32)
        amax = groups.abs().amax(2)
        m, e = torch.frexp(amax)
        # smallest 2^p with amax / 2^p <= 448 = 0.875 * 2^9
        p = torch.where(m <= 0.875, e - 9, e - 8).clamp(-127, 127)
        p = torch.where(amax > 0, p, torch.zeros_like(p))
        codes = torch.ldexp(groups, -p[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes = codes.view(T, H)
        scales = (p + 127).to(torch.uint8)
    return _norm_result(c, res, y.to(torch.bfloat16) if c["y"] else None, codes, scales)


def _linear_own(s, c):
    return _lib().linear(s["x"], s["w"], s["bias"],
                         activation=None if c["act"] == "none" else c["act"],
                         residual=s["residual"], out=s["out"])


def _linear_plain(s, c):
    v = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"]
    if c["act"] == "swiglu":
        gate, up = v[:, :c["N"]], v[:, c["N"]:]
        v = gate / (1 + torch.exp(-gate)) * up
    elif c["act"] == "silu":
        v = v / (1 + torch.exp(-v))
    elif c["act"] == "gelu":
        v = 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(_DT[c["out"]])


def _balance_own(s, c):
    moe = _lib()
    loss, counts, tokens, dlogits = moe.balance_loss(
        s["logits"], s["topk_ids"], COEF, c["scoring"], token_mask=s["mask"],
        seq_starts=s["seq_starts"], grad=c["mode"] == "fused", out=s["out"])
    if c["mode"] == "separate":
        dlogits = moe.balance_loss_backward(
            s["dloss"], s["logits"], counts, tokens, COEF, c["scoring"], token_mask=s["mask"],
            seq_starts=s["seq_starts"], out=s["out"][3])
    return _balance_result(loss, counts, tokens, dlogits if c["mode"] != "forward" else None)


def _balance_result(loss, counts, tokens, dlogits):
    out = {"loss": loss, "counts": counts, "tokens": tokens}
    if dlogits is not None:
        out["dlogits"] = dlogits
    return out


def _balance_plain(s, c):
    l = s["logits"].float()
    T, E = l.shape
    k, B = c["k"], c["B"]
    keep = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=l.device)
    if s["seq_starts"] is None:
        seq = torch.zeros(T, dtype=torch.int64, device=l.device)
    else:
        seq = torch.bucketize(torch.arange(T, device=l.device), s["seq_starts"][1:], right=True)
    # counts per (sequence, expert) and tokens per sequence
    counts = torch.zeros(B * E, dtype=torch.int64, device=l.device)
    flat = (seq[:, None] * E + s["topk_ids"]).reshape(-1)
    counts.index_add_(0, flat, keep[:, None].expand(T, k).reshape(-1).to(torch.int64))
    counts = counts.view(B, E)
    tokens = torch.zeros(B, dtype=torch.int64, device=l.device)
    tokens.index_add_(0, seq, keep.to(torch.int64))
    # scores, their derivative by the logit, and probabilities
    if c["scoring"] == "softmax":
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        dp = p
    else:
        sig = 1 / (1 + torch.exp(-l))
        if c["scoring"] == "sigmoid":
            score, dscore = sig, sig * (1 - sig)
        else:
            score = torch.sqrt(torch.clamp(l, min=0) + torch.log1p(torch.exp(-l.abs())))
            dscore = sig / (2 * score)
        total = score.sum(1, keepdim=True) + 1e-20
        p, dp = score / total, dscore / total
    # the load f = E * count / sum(count), less one: sum(p) = 1 takes the one
    # out of the gradient, and the difference is exact in whole numbers
    placed = counts.sum(1, keepdim=True)
    f1 = ((E * counts - placed).double() / placed.clamp(min=1)).float()
    some = tokens > 0
    share = torch.where(some, 1.0 / (some.sum() * tokens.clamp(min=1)).double(), 0.0).float()
    fr = f1[seq]
    mean = (fr * p).sum(1, keepdim=True)
    wt = (share[seq] * keep)[:, None] * COEF
    loss = (wt.double() * (1 + mean.double())).sum().float().view(1)
    dlogits = None
    if c["mode"] != "forward":
        dlogits = wt * dp * (fr - mean)
        if c["mode"] == "separate":
            dlogits = dlogits * s["dloss"]
        dlogits = dlogits.to(s["logits"].dtype)
    return _balance_result(loss, counts.to(torch.int32), tokens.to(torch.int32), dlogits)


# ---- the definitions in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        out = {}
        if s["residual"] is not None:
            h = h + s["residual"].double()
            out["residual"] = h
        rms = torch.sqrt((h * h).sum(1, keepdim=True) / case["H"] + EPS)
        y = h / rms * s["weight"].double()
        if case["y"]:
            out["y"] = y
        if case["e4m3"]:
            blocks = y.reshape(case["T"], -1, 32)
            big = blocks.abs().max(dim=2).values
            power = torch.where(big > 0, torch.ceil(torch.log2(big / 448)).clamp(-127, 127), 0.0)
            scale = torch.exp2(power)
            # what the codes approximate, before their rounding
            out["codes"] = (blocks / scale[..., None]).reshape(case["T"], case["H"])
            out["scales"] = scale
        return out
    if case["op"] == "linear":
        # in row blocks: the products of a whole prefill in 64 bits are large
        T, N, w = case["T"], case["N"], s["w"].double().t().contiguous()
        out = torch.empty((T, N), dtype=torch.float64, device="cuda")
        for r in range(0, T, 1024):
            z = torch.mm(s["x"][r:r + 1024].double(), w)
            if s["bias"] is not None:
                z += s["bias"].double()
            if case["act"] == "swiglu":
                a, b = z.split(N, dim=1)
                z = a * torch.sigmoid(a) * b
            elif case["act"] == "silu":
                z = z * torch.sigmoid(z)
            elif case["act"] == "gelu":
                z = z * torch.special.ndtr(z)
            if s["residual"] is not None:
                z = z + s["residual"][r:r + 1024].double()
            out[r:r + 1024] = z
        return out
    # the loss sequence by sequence, its gradient by automatic differentiation
    E, B = case["E"], case["B"]
    l = s["logits"].double().requires_grad_()
    if case["scoring"] == "softmax":
        p = torch.softmax(l, 1)
    else:
        sc = torch.sigmoid(l)
        if case["scoring"] == "sqrt_softplus":
            sc = torch.sqrt(-torch.nn.functional.logsigmoid(-l))
        p = sc / sc.sum(1, keepdim=True)
    bounds = [0, case["T"]] if s["seq_starts"] is None else s["seq_starts"].tolist()
    counts = torch.zeros((B, E), dtype=torch.int64, device="cuda")
    tokens = torch.zeros(B, dtype=torch.int64, device="cuda")
    terms = []
    for b in range(B):
        at = torch.arange(bounds[b], bounds[b + 1], device="cuda")
        if s["mask"] is not None:
            at = at[s["mask"][at]]
        tokens[b] = at.numel()
        if at.numel():
            counts[b] = torch.bincount(s["topk_ids"][at].reshape(-1).long(), minlength=E)
            f = counts[b].double() * E / (case["k"] * at.numel())
            terms.append((f * p[at].mean(0)).sum())
    loss = COEF * sum(terms) / max(1, len(terms)) + 0 * l.sum()
    dlogits = None
    if case["mode"] != "forward":
        dlogits, = torch.autograd.grad(loss, l)
        if case["mode"] == "separate":
            dlogits = dlogits * s["dloss"].double()
    return _balance_result(loss.detach().view(1), counts.to(torch.int32), tokens.to(torch.int32),
                           dlogits)


# ---- what a pass cannot do without ----------------------------------------------------

def work(case):
    size = {"bf16": 2, "f32": 4, "none": 0}
    if case["op"] == "norm":
        n = case["T"] * case["H"]
        b = n * (size[case["x"]] + 2 * size[case["res"]] + 2 * case["y"])
        b += case["H"] * size[case["w"]] + (n + n // 32 if case["e4m3"] else 0)
        return {"bytes": b, "flops": 5 * n}
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        rows = 2 * N if case["act"] == "swiglu" else N
        b = 2 * (T * K + rows * K) + T * N * (size[case["res"]] + size[case["out"]])
        return {"bytes": b + (4 * rows if case["bias"] else 0), "flops": 2 * T * K * rows}
    T, E, k, B = case["T"], case["E"], case["k"], case["B"]
    n = T * E * size[case["dt"]]
    # the gradient needs the loads of all tokens, so a separate backward reads
    # the logits a second time; one call reads them once
    b = {"forward": n, "fused": 2 * n, "separate": 3 * n}[case["mode"]]
    b += T * k * 4 + 4 * B * (E + 1) + (T if case["masked"] else 0)
    return {"bytes": b, "flops": 12 * T * E}
