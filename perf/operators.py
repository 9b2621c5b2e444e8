"""Measured cases of the operators that train one MoE layer's experts: the matrix products grouped
by expert (forward, input gradient, weight gradient), the SwiGLU activation with its routing weight
(forward and backward), and the AdamW step over many tensors.

`run` computes each case in its plain form (elementary torch operations in fp32), or, where `own` is
true, through the package's entry points.  `exact` computes the same outputs in 64 bits.
"""
import math

import torch

own = False
moe = None         # the package, imported where its operators are called

DEV = "cuda"
BLOCK = 128        # values that share one scale in the 8-bit optimiser states
TOP = 1.875        # the largest code stands for TOP * scale


def _moe():
    global moe
    if moe is None:
        import sparse_moe_layer_bailingmoev3_amd
        moe = sparse_moe_layer_bailingmoev3_amd
    return moe


# ---- cases -------------------------------------------------------------------------------------
# op "forward":  y[p] = W_g x[token of p]          (rows > 0 tokens T, top K of E experts, I x H weights)
# op "dgrad":    dx[p] = dy[p] W_g (+ dy2[p] W2_g)
# op "wgrad":    dW_g = sum over the group's positions of dy[p]^T x[p]
# `gather`: the operand is indexed by token (dispatch order comes from a row map), else by position.
# `skew`: popularity of the experts, 0 = uniform.

def _gemm(name, op, T, E, out_f, in_f, gather, fp32, acc=False, pair=False, skew=0.0, K=8):
    c = {"op": op, "T": T, "E": E, "K": K, "out_f": out_f, "in_f": in_f, "gather": gather, "fp32": fp32, "acc": acc,
         "pair": pair, "skew": skew}
    return {"name": name, **c} if name else c


def _swiglu(name, op, T, cols, limit, K=8):
    c = {"op": op, "T": T, "K": K, "cols": cols, "limit": limit}
    return {"name": name, **c} if name else c


def _adamw(name, tensors, rows, cols, vectors, vec, eight, master):
    c = {"op": "adamw", "tensors": tensors, "rows": rows, "cols": cols, "vectors": vectors, "vec": vec, "eight": eight,
         "master": master}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one token through the full layer's gate product: 8 experts, one row each (latency)
        _gemm("forward_gate_T1", "forward", 1, 512, 768, 2560, True, False),
        # a decode batch: about 325 of 512 experts with one to four rows (weights streamed once)
        _gemm("forward_gate_T64", "forward", 64, 512, 768, 2560, True, False),
        # the down product of a training step, written in fp32 for the combine
        _gemm("forward_down_T8192", "forward", 8192, 512, 2560, 768, False, True),
        # gradient of the activation: the output gradient gathered by token, times the down weights
        _gemm("dgrad_down_T8192", "dgrad", 8192, 512, 2560, 768, True, False),
        # gradient of the input through gate and up at once, skewed load, empty experts
        _gemm("dgrad_pair_skew_T4096", "dgrad", 4096, 512, 768, 2560, False, True, pair=True, skew=1.2),
        # weight gradient of the gate product added to the fp32 gradients of earlier micro-batches
        _gemm("wgrad_gate_acc_T8192", "wgrad", 8192, 512, 768, 2560, True, True, acc=True),
        # a small layer's weight gradient, sizes that fill no tile, skewed
        _gemm("wgrad_odd_T333", "wgrad", 333, 64, 136, 520, True, False, skew=0.8),
        # activation of a training step over all routed positions
        _swiglu("swiglu_T8192", "swiglu", 8192, 768, 4.0),
        # its gradient, with the gradient of the routing weights
        _swiglu("swiglu_backward_T8192", "swiglu_backward", 8192, 768, 4.0),
        # a short ragged batch of a small layer
        _swiglu("swiglu_backward_T97", "swiglu_backward", 97, 136, 0.0),
        # the expert weights of 128 experts, one tensor each as checkpoints hold them, states in 8 bits
        _adamw("adamw8_experts", 384, 768, 2560, 4, 2560, True, False),
        # a shared expert, router and vectors of odd length: fp32 states and master weights
        _adamw("adamw32_master", 6, 768, 2560, 48, 2559, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["forward", "dgrad", "wgrad", "swiglu", "swiglu_backward", "adamw"])
    if kind in ("forward", "dgrad", "wgrad"):
        E = rng.choice([64, 128, 256, 512])
        out_f, in_f = 8 * _log(rng, 8, 320), 8 * _log(rng, 16, 320)
        while out_f * in_f > 768 * 2560:
            out_f, in_f = 8 * _log(rng, 8, 320), 8 * _log(rng, 16, 320)
        fp32 = rng.random() < 0.5
        pair = kind == "dgrad" and rng.random() < 0.4
        return _gemm(None, kind, _log(rng, 1, 4096 if pair else 8192), E, out_f, in_f, rng.random() < 0.5, fp32,
                     acc=fp32 and rng.random() < 0.4, pair=pair,
                     skew=rng.choice([0.0, 0.0, 0.6, 1.2]), K=rng.choice([1, 4, 8]))
    if kind in ("swiglu", "swiglu_backward"):
        return _swiglu(None, kind, _log(rng, 1, 8192), 8 * _log(rng, 4, 96), rng.choice([0.0, 4.0, 7.0]), K=rng.choice([1, 8]))
    return _adamw(None, _log(rng, 1, 200), _log(rng, 16, 768), _log(rng, 16, 2560), _log(rng, 1, 64), _log(rng, 1, 4096),
                  rng.random() < 0.5, rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, scale=1.0):
    """bf16 normal values, drawn in pieces so that a large weight needs no fp32 copy."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV) * scale)
    return out


def _routing(case, g):
    """Top-K of noisy scores, grouped by expert: offsets [E+1], token of each position."""
    T, E, K = case["T"], case["E"], case["K"]
    popular = torch.randn(E, generator=g, device=DEV) * case["skew"]
    score = popular - torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEV).clamp(1e-9, 1 - 1e-6)))
    flat = score.topk(K, dim=1).indices.sort(dim=1).values.reshape(-1)
    order = torch.argsort(flat, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    return offsets, (order // K).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("forward", "dgrad", "wgrad"):
        T, E, N, K = case["T"], case["E"], case["out_f"], case["in_f"]
        offsets, token = _routing(case, g)
        P = token.numel()
        s = {"case": case, "offsets": offsets, "map": token if case["gather"] else None,
             "cap": int((offsets[1:] - offsets[:-1]).max())}  # the largest group, known to a program that pads
        dt = torch.float32 if case["fp32"] else torch.bfloat16
        rows = T if case["gather"] else P
        if op == "forward":
            s["x"], s["w"] = _randn(g, rows, K), _randn(g, E, N, K, scale=K ** -0.5)
            shape = (P, N)
        elif op == "dgrad":
            s["dy"], s["w"] = _randn(g, rows, N), _randn(g, E, N, K, scale=N ** -0.5)
            if case["pair"]:
                s["dy2"], s["w2"] = _randn(g, rows, N), _randn(g, E, N, K, scale=N ** -0.5)
            shape = (P, K)
        else:
            # gather: the token-indexed operand is x (gate and up), the gradient is by position
            s["dy"], s["x"] = _randn(g, P, N), _randn(g, rows, K)
            shape = (E, N, K)
        if case["acc"]:
            s["out"] = _randn(g, *shape).to(dt)
        else:
            s["out"] = torch.empty(shape, dtype=dt, device=DEV)
        return s
    if op in ("swiglu", "swiglu_backward"):
        P, C = case["T"] * case["K"], case["cols"]
        bf = dict(dtype=torch.bfloat16, device=DEV)
        s = {"case": case, "gate": _randn(g, P, C, scale=2.0), "up": _randn(g, P, C, scale=2.0),
             "row_w": torch.rand(P, generator=g, device=DEV) * 0.6 + 0.05,
             "pos": torch.randperm(P, generator=g, device=DEV).to(torch.int32)}
        if op == "swiglu":
            s["h"] = torch.empty((P, C), **bf)
        else:
            s["dh"] = _randn(g, P, C)
            s["dgate"], s["dup"] = torch.empty((P, C), **bf), torch.empty((P, C), **bf)
            s["drow_w"] = torch.empty(P, device=DEV)
        return s
    return _prepare_adamw(case, g)


def _sizes(case):
    """(numel, decayed) of every tensor: matrices decay, vectors do not."""
    return [case["rows"] * case["cols"]] * case["tensors"], [case["vec"]] * case["vectors"]


def _padded(n):
    return -(-n // BLOCK) * BLOCK


def _prepare_adamw(case, g):
    """All tensors lie in one arena (matrices, then vectors), each from a multiple of BLOCK values on."""
    mats, vecs = _sizes(case)
    cut = sum(map(_padded, mats))
    n = cut + sum(map(_padded, vecs))
    s = {"case": case, "cut": cut, "lr": 3e-4, "wd": 0.1, "step": 1000, "betas": (0.9, 0.999), "eps": 1e-8, "seed": 12345}
    p = _randn(g, n, scale=0.02)
    grad = _randn(g, n, scale=1e-3)
    m = _randn(g, n, scale=3e-4).float()
    v = _randn(g, n, scale=1e-3).float().square_().mul_(0.5).add_(1e-8)
    bounds, at = [], 0
    for size in mats + vecs:
        bounds.append((at, size))
        at += _padded(size)
    # the tail of a tensor's last block belongs to no tensor: zeros on both sides
    for a, size in bounds:
        if size % BLOCK:
            for t in (p, grad, m, v):
                t[a + size:a + _padded(size)] = 0
    s["p"], s["grad"] = p, grad
    s["master"] = p.float() if case["master"] else None
    rnd = _hash_base(bounds, n)
    s["rnd"] = rnd if case["eight"] else None
    if case["eight"]:
        s["m"], s["ms"] = _encode(m, rnd, s["seed"], 0, True)
        s["v"], s["vs"] = _encode(v, rnd, s["seed"], 0, False)
        s["mv"], s["vv"] = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    else:
        s["m"], s["v"] = m, v
    if own:  # the plan that a training program makes once and keeps
        cutouts = lambda t: [t[a:a + k] for a, k in bounds]  # noqa: E731
        scales = lambda t: [t[a // BLOCK:(a + _padded(k)) // BLOCK] for a, k in bounds]  # noqa: E731
        s["plan"] = _moe().MoEAdamWPlan(
            cutouts(p), cutouts(grad), cutouts(s["m"]), cutouts(s["v"]),
            master=cutouts(s["master"]) if case["master"] else None,
            exp_avg_scale=scales(s["ms"]) if case["eight"] else None,
            exp_avg_sq_scale=scales(s["vs"]) if case["eight"] else None,
            weight_decay=[s["wd"]] * len(mats) + [0.0] * len(vecs))
    return s


# ---- the 8-bit states --------------------------------------------------------------------------
# A block of 128 values shares scale = max|.| / 1.875.  With y = |.| / scale, a code c holds
# (1 + (c & 7) / 8) * 2^((c >> 3) - B): B = 15 and a sign in bit 7 for the first moment (code 0 is
# zero), B = 31 for the second.  Stochastic rounding: 16 bits of a hash of (seed, step, tensor,
# element) are added below the kept bits.

def _hash_base(bounds, n):
    """Per pair of values: (pair's index in its tensor, tensor's index), as the hash takes them."""
    tensor = torch.empty(n // 2, dtype=torch.int32, device=DEV)
    pair = torch.empty(n // 2, dtype=torch.int32, device=DEV)
    for i, (a, k) in enumerate(bounds):
        h = _padded(k) // 2
        tensor[a // 2:a // 2 + h] = i
        pair[a // 2:a // 2 + h] = torch.arange(h, device=DEV, dtype=torch.int32)
    return pair, tensor


def _bits16(rnd, seed, step):
    pair, tensor = rnd
    M = 0xFFFFFFFF
    key = (tensor.long() * 0x9E3779B9 + seed + step * 0x7F4A7C15) & M
    x = (pair.long() * 0x8DA6B343 + key) & M
    x ^= x >> 15
    x = (x * 0xD8163841) & M
    x ^= x >> 13
    x = (x * 0xCB1AB31F) & M
    x ^= x >> 16
    return torch.stack([x & 0xFFFF, x >> 16], 1).view(-1).to(torch.int32)


def _encode(t, rnd, seed, step, signed):
    b = t.view(-1, BLOCK)
    scale = b.abs().amax(1) * (1.0 / TOP)
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    inv = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
    y = (b.abs() * inv[:, None]).view(-1)
    bits = (y.view(torch.int32) + (_bits16(rnd, seed, step) << 4)) >> 20
    code = (bits - ((127 - (15 if signed else 31)) << 3)).clamp_(0, 127 if signed else 255)
    if signed:
        code |= (t < 0).int() << 7
    return code.to(torch.uint8), scale


def _decode(code, scale, signed):
    c = code.int()
    mag = c & 127 if signed else c
    y = ((mag << 20) + ((127 - (15 if signed else 31)) << 23)).view(torch.float32)
    if signed:
        y = torch.where(mag == 0, torch.zeros_like(y), torch.where(c > 127, -y, y))
    return (y.view(-1, BLOCK) * scale[:, None]).view(-1)


# ---- one pass ----------------------------------------------------------------------------------

def _groups(s, P):
    """Group of each position, and its place in the group's row of a padded batch."""
    p = torch.arange(P, device=DEV)
    gid = torch.searchsorted(s["offsets"][1:].long(), p, right=True)
    return gid, p - s["offsets"].long()[gid]


def _pad(s, a, mapped=True):
    """Rows of `a` by (group, place) in fp32, zeros where a group has fewer rows."""
    off = s["offsets"].long()
    p = off[:-1, None] + torch.arange(s["cap"], device=DEV)
    ok = p < off[1:, None]
    p = torch.where(ok, p, torch.zeros_like(p))
    r = s["map"].long()[p] if mapped and s["map"] is not None else p
    return torch.where(ok[..., None], a[r].float(), torch.zeros((), device=DEV))


def _rows(s, a):
    return a[s["map"].long()].float() if s["map"] is not None else a.float()


def _finish(s, y):
    if s["case"]["acc"]:
        return s["out"].add_(y)
    return y.to(s["out"].dtype)


def run(s):
    op = s["case"]["op"]
    return {"forward": _forward, "dgrad": _dgrad, "wgrad": _wgrad, "swiglu": _act, "swiglu_backward": _act_backward,
            "adamw": _step}[op](s)


def _forward(s):
    if own:
        _moe().moe_grouped_gemm(s["x"], s["w"], s["offsets"], s["out"], row_map=s["map"], accumulate=s["case"]["acc"])
        return s["out"]
    P, E = s["out"].shape[0], s["w"].shape[0]
    gid, place = _groups(s, P)
    if 4 * P <= E:  # few rows: each with a copy of its own expert's weights
        return _finish(s, (s["w"][gid].float() * _rows(s, s["x"])[:, None, :]).sum(2))
    y = torch.bmm(_pad(s, s["x"]), s["w"].float().transpose(1, 2).contiguous())
    return _finish(s, y.view(-1, y.shape[2])[gid * s["cap"] + place])


def _dgrad(s):
    if own:
        _moe().moe_grouped_gemm_dgrad(s["dy"], s["w"], s["offsets"], s["out"], row_map=s["map"], dy2=s.get("dy2"),
                                      w2=s.get("w2"), accumulate=s["case"]["acc"])
        return s["out"]
    P, E = s["out"].shape[0], s["w"].shape[0]
    gid, place = _groups(s, P)
    if 4 * P <= E:
        y = (s["w"][gid].float() * _rows(s, s["dy"])[:, :, None]).sum(1)
        if "dy2" in s:
            y = y + (s["w2"][gid].float() * _rows(s, s["dy2"])[:, :, None]).sum(1)
        return _finish(s, y)
    y = torch.bmm(_pad(s, s["dy"]), s["w"].float())
    if "dy2" in s:
        y = torch.baddbmm(y, _pad(s, s["dy2"]), s["w2"].float())
    return _finish(s, y.view(-1, y.shape[2])[gid * s["cap"] + place])


def _wgrad(s):
    if own:
        _moe().moe_grouped_gemm_wgrad(s["dy"], s["x"], s["offsets"], s["out"], x_map=s["map"], accumulate=s["case"]["acc"])
        return s["out"]
    dy = _pad(s, s["dy"], mapped=False)
    return _finish(s, torch.bmm(dy.transpose(1, 2).contiguous(), _pad(s, s["x"])))


def _act_parts(s):
    """Rows in the order of their routing weights; which values the clamp leaves (decided in 64 bits)."""
    pos = s["pos"].long()
    g, u = s["gate"][pos].float(), s["up"][pos].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    a = g * sig * u
    L = s["case"]["limit"]
    free = None
    if L > 0:
        gd = g.double()
        free = (gd / (1.0 + torch.exp(-gd)) * u.double()).abs() <= L
        a = torch.where(free, a, torch.sign(a) * L)
    return pos, g, u, sig, a, free


def _act(s):
    if own:
        _moe().moe_swiglu(s["gate"], s["up"], s["h"], limit=s["case"]["limit"], row_w=s["row_w"], pos=s["pos"])
        return s["h"]
    pos, _, _, _, a, _ = _act_parts(s)
    return torch.empty_like(s["h"]).index_copy_(0, pos, (a * s["row_w"][:, None]).bfloat16())


def _act_backward(s):
    if own:
        _moe().moe_swiglu_backward(s["gate"], s["up"], s["dh"], s["dgate"], s["dup"], limit=s["case"]["limit"],
                                   row_w=s["row_w"], pos=s["pos"], drow_w=s["drow_w"])
        return {"dgate": s["dgate"], "dup": s["dup"], "drow_w": s["drow_w"]}
    pos, g, u, sig, a, free = _act_parts(s)
    dh = s["dh"][pos].float()
    drow_w = (dh * a).sum(1)
    da = dh * s["row_w"][:, None]
    if free is not None:
        da = torch.where(free, da, torch.zeros_like(da))
    dgate = da * u * (sig * (1.0 + g * (1.0 - sig)))
    dup = da * (g * sig)
    back = lambda t: torch.empty_like(s["dgate"]).index_copy_(0, pos, t.bfloat16())  # noqa: E731
    return {"dgate": back(dgate), "dup": back(dup), "drow_w": drow_w}


def _step(s):
    case = s["case"]
    if own:
        _moe().moe_adamw_step(s["plan"], lr=s["lr"], step=s["step"], betas=s["betas"], eps=s["eps"], seed=s["seed"])
        if case["eight"]:
            _moe().moe_adamw_dequantise(s["m"], s["ms"], s["mv"], signed=True)
            _moe().moe_adamw_dequantise(s["v"], s["vs"], s["vv"], signed=False)
    else:
        b1, b2 = s["betas"]
        m = _decode(s["m"], s["ms"], True) if case["eight"] else s["m"]
        v = _decode(s["v"], s["vs"], False) if case["eight"] else s["v"]
        g = s["grad"].float()
        m = m * b1 + g * (1 - b1)
        v = v * b2 + g * g * (1 - b2)
        p = s["master"] if case["master"] else s["p"].float()
        # matrices first in the arena: they decay, the vectors behind them do not
        p = torch.cat([p[:s["cut"]] * (1 - s["lr"] * s["wd"]), p[s["cut"]:]])
        denom = (v * (1.0 / (1 - b2 ** s["step"]))).sqrt() + s["eps"]
        p = p - (s["lr"] / (1 - b1 ** s["step"])) * (m / denom)
        if case["master"]:
            s["master"].copy_(p)
        s["p"].copy_(p)
        if case["eight"]:
            s["m"], s["ms"] = _encode(m, s["rnd"], s["seed"], s["step"], True)
            s["v"], s["vs"] = _encode(v, s["rnd"], s["seed"], s["step"], False)
            s["mv"], s["vv"] = _decode(s["m"], s["ms"], True), _decode(s["v"], s["vs"], False)
        else:
            s["m"], s["v"] = m, v
    out = {"p": s["p"], "m": s["mv"] if case["eight"] else s["m"], "v": s["vv"] if case["eight"] else s["v"]}
    if case["master"]:
        out["master"] = s["master"]
    return out


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("forward", "dgrad", "wgrad"):
        T, E, K, N, D = case["T"], case["E"], case["K"], case["out_f"], case["in_f"]
        P = T * K
        touched = E * (1 - (1 - K / E) ** T)  # experts that a token reaches, uniform load
        size = 4 if case["fp32"] else 2
        twice = 2 if case["acc"] else 1
        pair = 2 if case["pair"] else 1
        rows = T if case["gather"] else P
        if op == "forward":
            b = touched * N * D * 2 + rows * D * 2 + P * N * size * twice
        elif op == "dgrad":
            b = pair * (touched * N * D * 2 + rows * N * 2) + P * D * size * twice
        else:
            b = P * N * 2 + rows * D * 2 + E * N * D * size * twice
        return {"bytes": float(b), "flops": 2.0 * P * N * D * pair}
    if op in ("swiglu", "swiglu_backward"):
        P, C = case["T"] * case["K"], case["cols"]
        planes = 3 if op == "swiglu" else 5
        return {"bytes": float(P * C * 2 * planes + P * 8), "flops": float(P * C * (8 if op == "swiglu" else 20))}
    n = sum(map(sum, _sizes(case)))
    per = 2 + 2 + 2 + (8 if case["master"] else 0)  # gradient, parameter in and out, master weights
    # 8 bits: codes and scales in and out, and the two moments read out as values
    per += 4 + 16 / BLOCK + 2 + 8 + 8 / BLOCK if case["eight"] else 16
    return {"bytes": float(n * per), "flops": float(n * 20)}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("forward", "dgrad", "wgrad"):
        at = s["offsets"].tolist()
        out = s["out"].double() if case["acc"] else torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            lo, hi = at[e], at[e + 1]
            if lo == hi:
                continue
            rows = s["map"][lo:hi].long() if s["map"] is not None else slice(lo, hi)
            if op == "forward":
                out[lo:hi] += s["x"][rows].double() @ s["w"][e].double().t()
            elif op == "dgrad":
                out[lo:hi] += s["dy"][rows].double() @ s["w"][e].double()
                if case["pair"]:
                    out[lo:hi] += s["dy2"][rows].double() @ s["w2"][e].double()
            else:
                out[e] += s["dy"][lo:hi].double().t() @ s["x"][rows].double()
        return out
    if op in ("swiglu", "swiglu_backward"):
        L = case["limit"]
        by_row = torch.empty(s["pos"].numel(), dtype=torch.float64, device=DEV)
        by_row[s["pos"].long()] = s["row_w"].double()  # weight of each matrix row
        g, u = s["gate"].double(), s["up"].double()
        sig = torch.sigmoid(g)
        a = g * sig * u
        inside = torch.ones_like(a) if L <= 0 else (a.abs() <= L).double()
        if L > 0:
            a = a.clamp(-L, L)
        if op == "swiglu":
            return a * by_row[:, None]
        dh = s["dh"].double()
        da = dh * by_row[:, None] * inside
        return {"dgate": da * u * sig * (1 + g - g * sig), "dup": da * g * sig, "drow_w": (dh * a).sum(1)[s["pos"].long()]}
    b1, b2 = s["betas"]
    t, lr = s["step"], s["lr"]
    m = (_decode(s["m"], s["ms"], True) if case["eight"] else s["m"]).double()
    v = (_decode(s["v"], s["vs"], False) if case["eight"] else s["v"]).double()
    g = s["grad"].double()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = (s["master"] if case["master"] else s["p"]).double()
    p[:s["cut"]] -= lr * s["wd"] * p[:s["cut"]]
    p -= lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + s["eps"])
    # a rounding to 8 bits has no value of its own in 64 bits: its codes hang on the last fp32 bit
    out = {"p": p, "m": None if case["eight"] else m, "v": None if case["eight"] else v}
    if case["master"]:
        out["master"] = p
    return out
