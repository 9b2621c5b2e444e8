"""Measured cases of the operators that train one MoE layer's router and prepare its step: the balance
loss with the experts' counts, the router's backward pass (gradients of the mixing weights and of the
balance loss to the logits, the router weight and the tokens), and the norm over many gradients with
its clipping.

`run` computes each case in its plain form (elementary torch operations in fp32), or, where `own` is
true, through the package's entry points.  `exact` computes the same outputs in 64 bits.
"""
import math

import torch

own = False
moe = None         # the package, imported where its operators are called

DEV = "cuda"
PAD = 128          # tensors of one arena of gradients begin at multiples of this
SCALE = 2.5        # routed_scaling_factor


def _moe():
    global moe
    if moe is None:
        import sparse_moe_layer_bailingmoev3_amd
        moe = sparse_moe_layer_bailingmoev3_amd
    return moe


# ---- cases -------------------------------------------------------------------------------------
# op "balance":   counts, mean scores and loss of T tokens in `seqs` sequences (`padded`: each ends in
#                 tokens that belong to none and were dispatched nowhere).  `skew`: popularity of experts.
# op "backward":  from the gradient of the mixing weights (`mix`) and of the balance loss (`balance`) to
#                 the logits (`dlogits`: returned), and, with `products`, to the router weight (`acc`: added
#                 to earlier micro-batches' gradients) and to the tokens (bf16, or added to fp32 rows).
# op "norm":      `big` tensors of rows x cols and `small` ones of `vec` values; `clip`: the clipped
#                 gradients are written too (as bf16).

def _balance(name, T, E, seqs, padded, skew, K=8):
    c = {"op": "balance", "T": T, "E": E, "K": K, "seqs": seqs, "padded": padded, "skew": skew}
    return {"name": name, **c} if name else c


def _backward(name, T, E, H, seqs, padded, mix=True, balance=True, products=True, dlogits=False, acc=False, dx32=False, norm=True, K=8):
    c = {"op": "backward", "T": T, "E": E, "H": H, "K": K, "seqs": seqs, "padded": padded, "mix": mix, "balance": balance,
         "products": products, "dlogits": dlogits, "acc": acc, "dx32": dx32, "norm": norm, "skew": 0.3}
    return {"name": name, **c} if name else c


def _norm(name, big, rows, cols, small, vec, fp32, clip):
    c = {"op": "norm", "big": big, "rows": rows, "cols": cols, "small": small, "vec": vec, "fp32": fp32, "clip": clip}
    return {"name": name, **c} if name else c


def listed():
    return [
        # the full layer's batch of a training step, one balance over all tokens
        _balance("balance_T8192", 8192, 512, 1, False, 0.3),
        # sixteen padded sequences of a larger batch, each balanced by itself, skewed load
        _balance("balance_seqs_T16384", 16384, 512, 16, True, 1.0),
        # a short ragged batch of a small layer (latency)
        _balance("balance_T61", 61, 64, 3, False, 0.3, K=4),
        # the router's whole backward pass of that training step, added to the layer's fp32 input gradient
        _backward("backward_T8192", 8192, 512, 2560, 1, False, dx32=True),
        # a few tokens (latency): only the mixing weights carry a gradient
        _backward("backward_T64", 64, 512, 2560, 1, False, balance=False),
        # a small layer, odd number of tokens in padded sequences, weight gradient added to earlier ones
        _backward("backward_seqs_T1333", 1333, 128, 640, 5, True, acc=True, dlogits=True),
        # weights frozen: the gradient of the logits alone
        _backward("dlogits_T16384", 16384, 256, 0, 16, False, products=False, dlogits=True),
        # gradients of 128 experts' weights, one tensor each as checkpoints hold them (the step takes the coefficient)
        _norm("norm_experts", 384, 768, 2560, 4, 2560, False, False),
        # fp32 gradients accumulated over micro-batches, clipped into the bf16 ones that a step reads
        _norm("clip_fp32", 48, 768, 2560, 50, 2559, True, True),
        # a router and vectors of odd length (latency)
        _norm("clip_router", 1, 512, 2560, 9, 513, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["balance", "backward", "backward", "norm"])
    if kind == "norm":
        fp32 = rng.random() < 0.5
        return _norm(None, _log(rng, 1, 96 if fp32 else 384), _log(rng, 16, 768), _log(rng, 16, 2560), _log(rng, 1, 64),
                     _log(rng, 1, 4096), fp32, rng.random() < 0.5)
    E, K, padded = rng.choice([64, 128, 256, 512, 1024]), rng.choice([1, 2, 4, 8]), rng.random() < 0.4
    if kind == "balance":
        T = _log(rng, 1, 8192 if E == 1024 else 16384)
        return _balance(None, T, E, _log(rng, 1, max(1, min(32, T // 2))), padded, rng.choice([0.0, 0.3, 1.0]), K=K)
    T, H = _log(rng, 1, 8192), 128 * rng.randint(1, 20)
    while T * E * H > 8192 * 512 * 2560:
        T, H = _log(rng, 1, 8192), 128 * rng.randint(1, 20)
    mix = rng.random() < 0.8
    return _backward(None, T, E, H, _log(rng, 1, max(1, min(32, T // 2))), padded, mix=mix, balance=not mix or rng.random() < 0.6,
                     dlogits=rng.random() < 0.3, acc=rng.random() < 0.4, dx32=rng.random() < 0.5, norm=K > 1 and rng.random() < 0.8, K=K)


# ---- inputs ------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _sequences(case, g):
    """(offsets [B+1], tokens of each sequence [B]): B cuts of T tokens, a padded one ends before its cut."""
    T, B = case["T"], case["seqs"]
    cuts = torch.rand(B - 1, generator=g, device=DEV).mul(T).long().sort().values
    edge = torch.tensor([0, T], device=DEV)
    off = torch.cat([edge[:1], cuts, edge[1:]])
    n = off[1:] - off[:-1]
    if case["padded"]:
        n = (n * (1 - 0.5 * torch.rand(B, generator=g, device=DEV))).ceil().long()
    return off.to(torch.int32), n.to(torch.int32)


def _config(case):
    groups = 8
    return _moe().MoEConfig(hidden_size=case.get("H") or 128, num_experts=case["E"], num_experts_per_tok=case["K"], n_group=groups,
                            topk_group=4, moe_intermediate_size=128, num_shared_experts=0, shared_intermediate_size=128,
                            norm_topk_prob=1 if case.get("norm", True) else 0, routed_scaling_factor=SCALE, swiglu_limit=0.0,
                            shared_swiglu_limit=0.0, expert_weight_format=0, expert_act_format=0)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "norm":
        return _prepare_norm(case, g)
    T, E, K = case["T"], case["E"], case["K"]
    s = {"case": case, "coef": 1e-3}
    if case.get("products"):
        H = case["H"]
        s["x"] = torch.randn(T, H, generator=g, device=DEV).bfloat16()
        s["rw"] = torch.randn(E, H, generator=g, device=DEV) * H ** -0.5
        s["logits"] = s["x"].float() @ s["rw"].t()
        s["drw"] = torch.randn(E, H, generator=g, device=DEV) * 1e-2
        s["dx"] = (torch.randn(T, H, generator=g, device=DEV) * 1e-2).to(torch.float32 if case["dx32"] else torch.bfloat16)
    else:
        s["logits"] = torch.randn(T, E, generator=g, device=DEV)
    popular = torch.randn(E, generator=g, device=DEV) * case["skew"]
    s["idx"] = (torch.sigmoid(s["logits"]) + 0.2 * popular).topk(K, dim=1).indices.sort(dim=1).values.to(torch.int32)
    s["off"], s["len"] = _sequences(case, g)
    at = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["off"][1:].long(), at, right=True)
    real = at - s["off"].long()[seq] < s["len"].long()[seq]
    s["idx"][~real] = -1
    s["padded"] = case["padded"]
    B = case["seqs"]
    if case["op"] == "balance":
        s["counts"] = torch.empty(B, E, dtype=torch.int32, device=DEV)
        s["probs"], s["loss"] = torch.empty(B, E, device=DEV), torch.empty(1, device=DEV)
    else:
        s["dw"] = torch.where(real[:, None], torch.randn(T, K, generator=g, device=DEV) * 1e-2, 0.0) if case["mix"] else None
        s["dloss"] = torch.rand(1, generator=g, device=DEV) + 0.5
        s["counts"] = torch.zeros(B * E, dtype=torch.int32, device=DEV)
        pairs = (seq[:, None] * E + s["idx"].long().clamp(min=0))[real].reshape(-1)
        s["counts"] = torch.bincount(pairs, minlength=B * E).view(B, E).to(torch.int32)
        s["dlogits"] = torch.empty(T, E, device=DEV)
    if own:
        s["cfg"] = _config(case)
        s["ws"] = torch.empty(_moe().moe_router_workspace_size(s["cfg"], T, B), dtype=torch.uint8, device=DEV)
    return s


def _prepare_norm(case, g):
    """All tensors lie in one arena, each from a multiple of PAD values on, zeros between them."""
    sizes = [case["rows"] * case["cols"]] * case["big"] + [case["vec"]] * case["small"]
    bounds, at = [], 0
    for n in sizes:
        bounds.append((at, n))
        at += -(-n // PAD) * PAD
    grad = torch.empty(at, dtype=torch.float32 if case["fp32"] else torch.bfloat16, device=DEV)
    for i in range(0, at, 1 << 28):
        part = grad[i:i + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV) * 1e-3)
    for a, n in bounds:
        grad[a + n:a + -(-n // PAD) * PAD] = 0
    s = {"case": case, "grad": grad, "scale": 0.25, "max": 0.1 * 0.25 * 1e-3 * math.sqrt(sum(sizes)),
         "norm": torch.empty(1, device=DEV), "coef": torch.empty(1, device=DEV)}
    if case["clip"]:
        s["out"] = torch.zeros(at, dtype=torch.bfloat16, device=DEV)
    if own:  # the plan that a training program makes once and keeps
        cut = lambda t: [t[a:a + n] for a, n in bounds]  # noqa: E731
        s["plan"] = _moe().MoEGradPlan(cut(grad), out=cut(s["out"]) if case["clip"] else None)
        s["ws"] = torch.empty(s["plan"].workspace_size, dtype=torch.uint8, device=DEV)
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    return {"balance": _run_balance, "backward": _run_backward, "norm": _run_norm}[s["case"]["op"]](s)


def _where(s):
    """Sequence of each token, whether it belongs to one, and both as fp32 rows of a [B,T] matrix."""
    T, B = s["logits"].shape[0], s["len"].numel()
    at = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["off"][1:].long(), at, right=True)
    real = at - s["off"].long()[seq] < s["len"].long()[seq]
    return seq, real, ((torch.arange(B, device=DEV)[:, None] == seq) & real).float()


def _scores(s):
    sig = 1.0 / (1.0 + torch.exp(-s["logits"]))
    return sig, sig / sig.sum(1, keepdim=True)


def _run_balance(s):
    case = s["case"]
    if own:
        _moe().moe_balance_loss(s["cfg"], case["T"], s["logits"], s["idx"], s["coef"], s["counts"], s["probs"], s["loss"], s["ws"],
                                seq_offsets=s["off"], seq_lens=s["len"] if s["padded"] else None)
        return {"counts": s["counts"], "probs": s["probs"], "loss": s["loss"]}
    E, K, B = case["E"], case["K"], case["seqs"]
    seq, real, member = _where(s)
    n = s["len"].float()
    idx = s["idx"].long()
    ok = real[:, None] & (idx >= 0) & (idx < E)
    # pairs that count nowhere go to one entry more
    pair = torch.where(ok, seq[:, None] * E + idx, torch.full_like(idx, B * E)).reshape(-1)
    ones = torch.ones(pair.numel(), dtype=torch.int32, device=DEV)
    counts = torch.zeros(B * E + 1, dtype=torch.int32, device=DEV).scatter_add_(0, pair, ones)[:-1].view(B, E)
    probs = (member @ _scores(s)[1]) / n.clamp(min=1)[:, None]
    # n_b / N * E / (K n_b) of every sequence alike
    loss = (counts.float() * probs).sum() * (s["coef"] * E / K) / n.sum()
    return {"counts": counts, "probs": probs, "loss": loss.view(1)}


def _dlogits(s):
    case = s["case"]
    E, K = case["E"], case["K"]
    sig, p = _scores(s)
    d = torch.zeros_like(sig)
    if case["balance"]:
        seq, real, _ = _where(s)
        n = s["len"].float()
        f = (s["counts"].float() * (E / K) / n.clamp(min=1)[:, None])[seq]
        d = (f - (f * p).sum(1, keepdim=True)) * p * (1 - sig) * (s["dloss"] * s["coef"] / n.sum())
        d = torch.where(real[:, None], d, torch.zeros_like(d))
    if case["mix"]:
        ok = s["idx"] >= 0
        at = s["idx"].long().clamp(min=0)
        zero = torch.zeros_like(s["dw"])
        sk = torch.where(ok, sig.gather(1, at), zero)
        gk = torch.where(ok, s["dw"] * SCALE, zero)
        if case["norm"]:
            q = sk / sk.sum(1, keepdim=True)
            gk = torch.where(ok, (gk - (gk * q).sum(1, keepdim=True)) * q * (1 - sk), zero)
        else:
            gk = gk * sk * (1 - sk)
        d.scatter_add_(1, at, gk)
    return d


def _run_backward(s):
    case = s["case"]
    if own:
        prod = case["products"]
        _moe().moe_router_backward(
            s["cfg"], case["T"], s["logits"], s["idx"], dtopk_w=s["dw"], counts=s["counts"] if case["balance"] else None,
            coef=s["coef"], dloss=s["dloss"], seq_offsets=s["off"], seq_lens=s["len"] if s["padded"] else None,
            dlogits=s["dlogits"] if case["dlogits"] else None, x=s["x"] if prod else None, router_w=s["rw"] if prod else None,
            drouter_w=s["drw"] if prod else None, accumulate_w=case["acc"], dx=s["dx"] if prod else None, accumulate_x=case["dx32"],
            ws=s["ws"])
        out = {"drouter_w": s["drw"], "dx": s["dx"]} if prod else {}
        return {**out, "dlogits": s["dlogits"]} if case["dlogits"] else out
    d, out = _dlogits(s), {}
    if case["products"]:
        dw, dx = d.t() @ s["x"].float(), d @ s["rw"]
        out["drouter_w"] = s["drw"].add_(dw) if case["acc"] else dw
        out["dx"] = s["dx"].add_(dx) if case["dx32"] else dx.bfloat16()
    return {**out, "dlogits": d} if case["dlogits"] else out


def _run_norm(s):
    clip = s["case"]["clip"]
    if own:
        _moe().moe_grad_norm(s["plan"], s["max"], s["norm"], s["coef"], s["ws"], scale=s["scale"])
        if clip:
            _moe().moe_grad_clip(s["plan"], s["coef"])
        return {"norm": s["norm"], "coef": s["coef"], **({"out": s["out"]} if clip else {})}
    g = s["grad"].float()
    norm = s["scale"] * (g * g).sum(dtype=torch.float64).sqrt()
    coef = s["scale"] * torch.where(norm <= s["max"], torch.ones_like(norm), s["max"] / norm)
    norm, coef = norm.float().view(1), coef.float().view(1)
    return {"norm": norm, "coef": coef, **({"out": (g * coef).bfloat16()} if clip else {})}


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    if case["op"] == "norm":
        n = case["big"] * case["rows"] * case["cols"] + case["small"] * case["vec"]
        size = 4 if case["fp32"] else 2
        return {"bytes": float(n * (size + (2 if case["clip"] else 0))), "flops": float(n * (3 if case["clip"] else 2))}
    T, E, K = case["T"], case["E"], case["K"]
    if case["op"] == "balance":
        return {"bytes": float(T * E * 4 + T * K * 4 + case["seqs"] * E * 8), "flops": float(T * E * 6)}
    b, f = T * E * 4 + T * K * 4 + (T * K * 4 if case["mix"] else 0), T * E * 10.0
    if case["balance"]:
        b += case["seqs"] * E * 4
    if case["dlogits"]:
        b += T * E * 4
    if case["products"]:
        H = case["H"]
        b += T * H * 2 + E * H * 4 + E * H * 4 * (2 if case["acc"] else 1) + T * H * (8 if case["dx32"] else 2)
        f += 4.0 * T * E * H
    return {"bytes": float(b), "flops": float(f)}


# ---- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        total = 0.0
        for part in s["grad"].split(1 << 26):
            total += float((part.double() ** 2).sum())
        norm = s["scale"] * math.sqrt(total)
        coef = s["scale"] * min(1.0, s["max"] / norm)
        as64 = lambda v: torch.tensor([v], dtype=torch.float64, device=DEV)  # noqa: E731
        return {"norm": as64(norm), "coef": as64(coef), **({"out": s["grad"].double() * coef} if case["clip"] else {})}
    E, K, B, T = case["E"], case["K"], case["seqs"], case["T"]
    sig = torch.sigmoid(s["logits"].double())
    off, n, idx = s["off"].tolist(), s["len"].tolist(), s["idx"].long()
    N = sum(n)
    if case["op"] == "balance":
        counts = torch.zeros(B, E, dtype=torch.int32, device=DEV)
        probs, loss = torch.zeros(B, E, dtype=torch.float64, device=DEV), 0.0
        for b in range(B):
            if n[b] == 0:
                continue
            rows = slice(off[b], off[b] + n[b])
            chosen = idx[rows].reshape(-1)
            counts[b] = torch.bincount(chosen[chosen >= 0], minlength=E).to(torch.int32)
            probs[b] = torch.nn.functional.normalize(sig[rows], p=1, dim=1).mean(0)
            load = counts[b].double() * E / (K * n[b])
            loss += n[b] / N * float(load @ probs[b])
        return {"counts": counts, "probs": probs, "loss": torch.tensor([s["coef"] * loss], dtype=torch.float64, device=DEV)}
    # the derivative with respect to the scores, then through the sigmoid
    ds = torch.zeros_like(sig)
    if case["balance"]:
        for b in range(B):
            rows = slice(off[b], off[b] + n[b])
            load = s["counts"][b].double() * E / max(1, K * n[b])
            total = sig[rows].sum(1, keepdim=True)
            ds[rows] = s["dloss"].double() * s["coef"] / max(N, 1) * (load / total - (sig[rows] @ load)[:, None] / total ** 2)
    if case["mix"]:
        rows = torch.nonzero(idx[:, 0] >= 0)[:, 0]
        at, gk = idx[rows], s["dw"][rows].double() * SCALE
        if case["norm"]:
            sk = sig[rows].gather(1, at)
            total = sk.sum(1, keepdim=True)
            gk = gk / total - (gk * sk).sum(1, keepdim=True) / total ** 2
        part = ds[rows]
        ds[rows] = part.scatter_add(1, at, gk)
    d = ds * sig * (1 - sig)
    out = {}
    if case["products"]:
        dw, dx = d.t().contiguous() @ s["x"].double(), d @ s["rw"].double()
        out["drouter_w"] = dw + s["drw"].double() if case["acc"] else dw
        out["dx"] = dx + s["dx"].double() if case["dx32"] else dx
    return {**out, "dlogits": d} if case["dlogits"] else out
