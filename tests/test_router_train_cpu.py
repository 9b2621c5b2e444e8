"""The operators that train the router, and the gradient norm, without a GPU: their definitions, and what
the host layer and the binding refuse before anything is enqueued (addresses given here are never
dereferenced)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import sparse_moe_layer_bailingmoev3_amd as moe
from oracle import router_oracle as orc

needs_lib = pytest.mark.skipif(not os.path.exists(moe.lib_path()), reason="libmoe.so not built")

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = -1, -2, -3, -4
A = 1 << 40                                # an aligned address
BIG = 1 << 34                              # bytes of workspace, enough for every size below


def at(i):
    return A + (i << 36)                   # far enough apart for every size below


def config(E=64, K=4, H=128, **kw):
    d = dict(hidden_size=H, num_experts=E, num_experts_per_tok=K, n_group=8, topk_group=4, moe_intermediate_size=128,
             num_shared_experts=0, shared_intermediate_size=128, norm_topk_prob=1, routed_scaling_factor=2.5)
    d.update(kw)
    return moe.MoEConfig(**d)


def seqs(**kw):
    d = dict(n_seq=3, offsets=at(20), lens=None)
    d.update(kw)
    return moe._Sequences(**d)


def balance(cfg=None, T=100, seq=None, logits=at(1), idx=at(2), coef=1.0, counts=at(3), probs=at(4), loss=at(5), ws=at(6), n=BIG):
    cfg = cfg or config()
    return moe.load_library().moe_balance_loss(ctypes.byref(cfg), T, ctypes.byref(seq) if seq else None, logits, idx, coef, counts, probs,
                                               loss, ws, n, None)


def backward(cfg=None, T=100, seq=None, ws=at(6), n=BIG, none=False, **kw):
    cfg = cfg or config()
    d = dict(logits=at(1), topk_idx=at(2), dtopk_w=at(3), counts=at(4), balance_coef=1.0, dloss=None, x=at(7), router_w=at(8),
             dlogits=at(9), drouter_w=at(10), accumulate_w=0, dx=at(11), dx_dtype=0, accumulate_x=0)
    d.update(kw)
    g = moe._RouterBackward(**d)
    return moe.load_library().moe_router_backward(ctypes.byref(cfg), T, ctypes.byref(seq) if seq else None,
                                                  None if none else ctypes.byref(g), ws, n, None)


def route(T=100, logits=at(5), idx=at(3), cfg=None, ws=at(6), n=BIG):
    cfg = cfg or config()
    return moe.load_library().moe_route_logits(ctypes.byref(cfg), T, at(1), at(2), None, idx, at(4), logits, ws, n, None)


@needs_lib
@pytest.mark.parametrize("call,code,words", [
    (lambda: balance(config(E=100)), UNSUPPORTED, b"num_experts"),
    (lambda: balance(T=-1), INVALID, b"T = -1"),
    (lambda: balance(T=2**31 // 5 + 1), UNSUPPORTED, b"32-bit"),
    (lambda: balance(seq=seqs(n_seq=0)), INVALID, b"n_seq 0"),
    (lambda: balance(seq=seqs(n_seq=65537)), UNSUPPORTED, b"above 65536"),
    (lambda: balance(seq=seqs(offsets=None)), INVALID, b"need offsets"),
    (lambda: balance(seq=seqs(offsets=at(20) + 2)), ALIGNMENT, b"sequence offsets"),
    (lambda: balance(seq=seqs(lens=at(21) + 1)), ALIGNMENT, b"sequence lens"),
    (lambda: balance(coef=float("nan")), INVALID, b"coef"),
    (lambda: balance(logits=None), INVALID, b"logits"),
    (lambda: balance(logits=at(1) + 4), ALIGNMENT, b"logits"),
    (lambda: balance(idx=None), INVALID, b"topk_idx"),
    (lambda: balance(counts=None), INVALID, b"counts"),
    (lambda: balance(probs=at(4) + 8), ALIGNMENT, b"probs"),
    (lambda: balance(loss=None), INVALID, b"loss"),
    (lambda: balance(ws=None), WORKSPACE, b"workspace"),
    (lambda: balance(ws=at(6) + 16), ALIGNMENT, b"workspace"),
    (lambda: balance(n=100), WORKSPACE, b"100 bytes"),
    (lambda: balance(counts=at(1) + 25600 - 16), INVALID, b"counts overlaps logits"),
    (lambda: balance(probs=at(3)), INVALID, b"probs overlaps counts"),
    (lambda: balance(loss=at(2) + 64), INVALID, b"loss overlaps topk_idx"),
    (lambda: balance(ws=at(4)), INVALID, b"workspace overlaps probs"),
    (lambda: balance(seq=seqs(offsets=at(3) + 8)), INVALID, b"counts overlaps sequence offsets"),
    (lambda: balance(seq=seqs(lens=at(5))), INVALID, b"loss overlaps sequence lens"),
    (lambda: backward(none=True), INVALID, b"gradients"),
    (lambda: backward(dtopk_w=None, counts=None), INVALID, b"dtopk_w or counts"),
    (lambda: backward(dlogits=None, drouter_w=None, dx=None), INVALID, b"dlogits, drouter_w or dx"),
    (lambda: backward(balance_coef=float("inf")), INVALID, b"balance_coef"),
    (lambda: backward(dx_dtype=2), INVALID, b"dtype 2"),
    (lambda: backward(accumulate_x=1), UNSUPPORTED, b"accumulation needs fp32"),
    (lambda: backward(config(H=65536 + 128)), UNSUPPORTED, b"hidden_size"),
    (lambda: backward(logits=None), INVALID, b"logits"),
    (lambda: backward(topk_idx=None), INVALID, b"topk_idx"),
    (lambda: backward(x=None), INVALID, b"x must not be NULL"),
    (lambda: backward(router_w=None), INVALID, b"router_w must not be NULL"),
    (lambda: backward(dtopk_w=at(3) + 4), ALIGNMENT, b"dtopk_w"),
    (lambda: backward(counts=at(4) + 4), ALIGNMENT, b"counts"),
    (lambda: backward(dloss=at(12) + 2), ALIGNMENT, b"dloss"),
    (lambda: backward(dx=at(11) + 8), ALIGNMENT, b"dx"),
    (lambda: backward(ws=None), WORKSPACE, b"workspace"),
    (lambda: backward(n=1000), WORKSPACE, b"1000 bytes"),
    (lambda: backward(dlogits=at(1)), INVALID, b"dlogits overlaps logits"),
    (lambda: backward(drouter_w=at(8)), INVALID, b"drouter_w overlaps router_w"),
    (lambda: backward(dx=at(7)), INVALID, b"dx overlaps x"),
    (lambda: backward(dx=at(9) + 16), INVALID, b"dx overlaps dlogits"),
    (lambda: backward(drouter_w=at(3) + 1600 - 16), INVALID, b"drouter_w overlaps dtopk_w"),
    (lambda: backward(ws=at(10)), INVALID, b"workspace overlaps drouter_w"),
    (lambda: backward(dloss=at(11) + 16), INVALID, b"dx overlaps dloss"),
    (lambda: backward(seq=seqs(lens=at(9))), INVALID, b"dlogits overlaps sequence lens"),
    (lambda: route(logits=None), INVALID, b"logits"),
    (lambda: route(logits=at(5) + 8), ALIGNMENT, b"logits"),
    (lambda: route(idx=None), INVALID, b"topk_idx"),
    (lambda: route(n=10), WORKSPACE, b"10 bytes"),
])
def test_router_refusals(call, code, words):
    assert call() == code
    assert words in moe.load_library().moe_last_error()


def route_logits(T=100, **kw):
    d = dict(x=at(1), router_w=at(2), bias=at(7), idx=at(3), w=at(4), logits=at(5), ws=at(6))
    d.update(kw)
    return moe.load_library().moe_route_logits(ctypes.byref(config()), T, d["x"], d["router_w"], d["bias"], d["idx"], d["w"], d["logits"],
                                               d["ws"], BIG, None)


@needs_lib
@pytest.mark.parametrize("given,words", [
    (dict(logits=at(1)), b"logits overlaps x"), (dict(logits=at(2) + 64 * 128 * 4 - 16), b"logits overlaps router_w"),
    (dict(bias=at(5) + 256), b"logits overlaps expert_bias"), (dict(idx=at(1) + 16), b"topk_idx overlaps x"),
    (dict(w=at(2)), b"topk_w overlaps router_w"), (dict(w=at(3) + 16), b"topk_w overlaps topk_idx"),
    (dict(logits=at(3)), b"logits overlaps topk_idx"), (dict(logits=at(4) + 1600 - 16), b"logits overlaps topk_w"),
    (dict(ws=at(1)), b"workspace overlaps x"), (dict(logits=at(6)), b"workspace overlaps logits"),
    (dict(idx=at(6) + 512), b"workspace overlaps topk_idx"), (dict(router_w=at(6) + 256), b"workspace overlaps router_w"),
], ids=str)
def test_route_logits_refuses_overlaps(given, words):
    assert route_logits(**given) == INVALID
    assert words in moe.load_library().moe_last_error()


@needs_lib
def test_workspace_size():
    cfg = config(E=512, K=8, H=2560)
    assert moe.moe_router_workspace_size(cfg, 0) > 0
    a, b = moe.moe_router_workspace_size(cfg, 64), moe.moe_router_workspace_size(cfg, 8192)
    assert a < b
    assert moe.moe_router_workspace_size(cfg, 64, 4096) > 4096 * 512 * 8   # a row of sums and counts a sequence
    for bad in (0, 65537):
        with pytest.raises(moe.MoEError):
            moe.moe_router_workspace_size(cfg, 64, bad)


@needs_lib
@pytest.mark.parametrize("E,H", [(64, 128), (64, 2560), (128, 640), (512, 2560), (1024, 128), (1024, 4096)])
def test_workspace_size_never_falls(E, H):
    cfg = config(E=E, H=H)
    edges = [32 * i + d for i in range(300) for d in (0, 1)] + [c * n + d for c in (4, 8, 16, 32, 64, 128, 256) for n in (1, 7, 256, 1000)
                                                               for d in (-1, 0, 1)]
    Ts = sorted({*edges, *range(0, 70000, 997), 10**6, 10**7})
    before = None
    for n in (1, 2, 7, 64, 65, 1000, 65536):
        sizes = [moe.moe_router_workspace_size(cfg, T, n) for T in Ts]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), [t for t, a, b in zip(Ts[1:], sizes, sizes[1:]) if a > b][:3]
        assert before is None or all(a <= b for a, b in zip(before, sizes))
        before = sizes


@needs_lib
@pytest.mark.parametrize("E,H", [(64, 128), (128, 640), (512, 2560), (1024, 256)])
def test_workspace_for_the_longest_batch_serves_every_shorter_one(E, H):
    """A call that a workspace satisfies goes on to the next check: here, that an output lies on an input."""
    cfg = config(E=E, H=H)
    for T, n in ((2000, 3), (8200, 40), (33000, 1), (70000, 300)):
        size = moe.moe_router_workspace_size(cfg, T, n)
        for t in sorted({*range(1, T + 1, max(1, T // 400)), *(c * 256 for c in (32, 64, 128) if c * 256 <= T), T}):
            q = seqs(n_seq=n) if n > 1 else None
            # (addresses of one sequence and of n: apart from each other for every size here)
            assert balance(cfg, t, q, probs=at(1), n=size) == INVALID
            for kw in (dict(), dict(dx=None), dict(drouter_w=None), dict(dx_dtype=1)):
                assert backward(cfg, t, q, dlogits=at(1), n=size, **kw) == INVALID


# ---- norm ------------------------------------------------------------------------------------------

def grad_plan(tensors, image=None, n=0, plan=True, count=None):
    table = (moe._GradTensor * max(1, len(tensors)))(*tensors)
    p = moe._GradPlan()
    st = moe.load_library().moe_grad_plan(len(tensors) if count is None else count, ctypes.byref(table) if tensors else None,
                                          ctypes.byref(p) if plan else None, image, n)
    return st, p


def tensor(i=1, out=None, numel=100, grad_dtype=0, out_dtype=0, off=0):
    return moe._GradTensor(at(i) + off, out, numel, grad_dtype, out_dtype)


def planned(*tensors):
    """With an image, where overlaps are looked for."""
    buf = ctypes.create_string_buffer(1 << 16)
    return grad_plan(tensors, ctypes.addressof(buf), 1 << 16)[0]


@needs_lib
@pytest.mark.parametrize("call,code,words", [
    (lambda: grad_plan([tensor()], plan=False)[0], INVALID, b"plan"),
    (lambda: grad_plan([], count=-1)[0], INVALID, b"n_tensors"),
    (lambda: grad_plan([], count=3)[0], INVALID, b"tensors must not be NULL"),
    (lambda: planned(tensor(grad_dtype=5)), INVALID, b"dtype 5"),
    (lambda: planned(tensor(numel=-1)), INVALID, b"numel = -1"),
    (lambda: planned(tensor(numel=(1 << 40) + 1)), UNSUPPORTED, b"too large"),
    (lambda: planned(tensor(off=8)), ALIGNMENT, b"tensor 0: grad"),
    (lambda: planned(moe._GradTensor(None, None, 5, 0, 0)), INVALID, b"tensor 0: grad must not be NULL"),
    (lambda: planned(tensor(), tensor(2, out=at(3) + 2)), ALIGNMENT, b"tensor 1: out"),
    (lambda: planned(tensor(out_dtype=1)), INVALID, b"keeps its type"),
    (lambda: planned(tensor(out=at(1), out_dtype=1)), INVALID, b"keeps its type"),
    (lambda: planned(tensor(), tensor(off=192)), INVALID, b"overlaps another"),
    (lambda: planned(tensor(out=at(2)), tensor(3, out=at(2))), INVALID, b"overlaps another"),
    (lambda: planned(tensor(out=at(2)), tensor(2, out=at(3))), INVALID, b"overlaps another"),
    (lambda: planned(tensor(out=at(1) + 16)), INVALID, b"overlaps another"),
])
def test_grad_plan_refusals(call, code, words):
    assert call() == code
    assert words in moe.load_library().moe_last_error()


@needs_lib
def test_grad_plan_takes_what_is_apart():
    # two gradients that are only read may be one array; empty ones have no address
    assert planned(tensor(out=at(2)), tensor(out=at(3)), moe._GradTensor(None, None, 0, 0, 0)) == 0
    assert planned(tensor(numel=128), tensor(numel=128, off=256)) == 0
    st, p = grad_plan([tensor(numel=100), tensor(2, numel=20000)])
    assert st == 0 and p.n_chunks == 1 + 3 and p.n_tensors == 2 and p.workspace_bytes > 0
    buf = ctypes.create_string_buffer(p.image_bytes)
    assert grad_plan([tensor(numel=100), tensor(2, numel=20000)], ctypes.addressof(buf), p.image_bytes - 1)[0] == WORKSPACE


def norm(plan=None, image=at(1), max_norm=1.0, scale=1.0, out=at(2), coef=at(3), ws=at(4), n=1 << 20):
    p = plan if plan is not None else grad_plan([tensor(9)])[1]
    return moe.load_library().moe_grad_norm(ctypes.byref(p), image, max_norm, scale, out, coef, ws, n, None)


@needs_lib
@pytest.mark.parametrize("call,code,words", [
    (lambda: moe.load_library().moe_grad_norm(None, at(1), 1.0, 1.0, at(2), at(3), at(4), 1 << 20, None), INVALID, b"plan"),
    (lambda: norm(moe._GradPlan(1, -1, 0, 0)), INVALID, b"plan"),
    (lambda: norm(image=None), INVALID, b"image"),
    (lambda: norm(image=at(1) + 8), ALIGNMENT, b"image"),
    (lambda: norm(max_norm=-1.0), INVALID, b"max_norm"),
    (lambda: norm(max_norm=float("nan")), INVALID, b"max_norm"),
    (lambda: norm(scale=float("inf")), INVALID, b"scale"),
    (lambda: norm(out=None), INVALID, b"norm"),
    (lambda: norm(out=at(2) + 2), ALIGNMENT, b"norm"),
    (lambda: norm(coef=at(3) + 1), ALIGNMENT, b"coef"),
    (lambda: norm(coef=at(2)), INVALID, b"coef overlaps norm"),
    (lambda: norm(out=at(4) + 8), INVALID, b"workspace overlaps norm"),
    (lambda: norm(out=at(1) + 4), INVALID, b"norm overlaps image"),
    (lambda: norm(ws=None), WORKSPACE, b"workspace"),
    (lambda: norm(n=1000), WORKSPACE, b"1000 bytes"),
    (lambda: moe.load_library().moe_grad_clip(ctypes.byref(grad_plan([tensor()])[1]), at(1), None, None), INVALID, b"coef"),
    (lambda: moe.load_library().moe_grad_clip(ctypes.byref(grad_plan([tensor()])[1]), None, at(3), None), INVALID, b"image"),
])
def test_grad_norm_refusals(call, code, words):
    assert call() == code
    assert words in moe.load_library().moe_last_error()


# ---- the binding -------------------------------------------------------------------------------------

def cpu_args(T=10, E=64, K=4, H=128):
    z = torch.zeros
    return dict(logits=z(T, E), topk_idx=z(T, K, dtype=torch.int32), dtopk_w=z(T, K), counts=z(1, E, dtype=torch.int32),
                x=z(T, H, dtype=torch.bfloat16), router_w=z(E, H), dlogits=z(T, E), drouter_w=z(E, H), dx=z(T, H),
                ws=z(100, dtype=torch.uint8))


@needs_lib
@pytest.mark.parametrize("name,value,words", [
    ("logits", torch.zeros(10, 65), "logits is"), ("logits", torch.zeros(10, 64, dtype=torch.float64), "logits must be"),
    ("logits", 3, "logits must be a tensor"), ("topk_idx", torch.zeros(10, 4, dtype=torch.int64), "topk_idx must be"),
    ("dtopk_w", torch.zeros(9, 4), "dtopk_w is"), ("dtopk_w", torch.zeros(4, 10).t(), "dtopk_w must be contiguous"),
    ("counts", torch.zeros(2, 64, dtype=torch.int32), "counts is"), ("x", torch.zeros(10, 128), "x must be"),
    ("x", None, "drouter_w needs x"), ("router_w", None, "dx needs router_w"), ("router_w", torch.zeros(64), "2 dimension"),
    ("drouter_w", torch.zeros(64, 256)[:, ::2], "contiguous"), ("dx", torch.zeros(10, 128, dtype=torch.float16), "dx must be"),
    ("dx", "dx", "dx must be a tensor"), ("ws", [1], "ws must be"), ("dloss", torch.zeros(2), "dloss must hold"),
    ("seq_lens", torch.zeros(3, dtype=torch.int32), "seq_lens has 3"), ("seq_offsets", torch.zeros(3), "seq_offsets must be"),
    ("cfg", None, "cfg must be"), (None, None, "must lie on a GPU"),
], ids=str)
def test_binding_refusals(name, value, words):
    args, cfg = cpu_args(), config()
    if name == "cfg":
        cfg = value
    elif name is not None:
        args[name] = value
    logits, idx = args.pop("logits"), args.pop("topk_idx")
    with pytest.raises(moe.MoEError, match=words):
        moe.moe_router_backward(cfg, 10, logits, idx, **args)


@needs_lib
def test_binding_refuses_plans():
    z = torch.zeros(5)
    for call, words in ((lambda: moe.MoEGradPlan([]), "must not be empty"), (lambda: moe.MoEGradPlan(3), "lists of tensors"),
                        (lambda: moe.MoEGradPlan([z], out=[]), "out has 0"), (lambda: moe.MoEGradPlan([1]), "must be a tensor"),
                        (lambda: moe.MoEGradPlan([z]), "one GPU"), (lambda: moe.moe_grad_norm(1, 1.0, z, z, z), "MoEGradPlan"),
                        (lambda: moe.moe_grad_clip(None, z), "MoEGradPlan")):
        with pytest.raises(moe.MoEError, match=words):
            call()


# ---- the definitions -------------------------------------------------------------------------------

@pytest.mark.parametrize("norm", [0, 1])
def test_oracle_gradient_against_differences(norm):
    rng = np.random.default_rng(1)
    T, E, K = 9, 64, 4
    logits, dw = rng.normal(size=(T, E)) * 2, rng.normal(size=(T, K))
    idx = np.sort(np.argsort(rng.random((T, E)), 1)[:, :K], 1)
    idx[3] = -1
    off, lens = [1, 4, 4, 8], [2, 5, 4]
    counts = orc.balance_loss(logits, idx, K, 1.0, off, lens).counts

    def loss(l):
        s = 1 / (1 + np.exp(-l))
        total = 0.0
        for t in range(T):
            if idx[t, 0] >= 0:
                sk = s[t, idx[t]]
                total += (2.5 * sk / (sk.sum() if norm else 1.0) * dw[t]).sum()
        p = s / s.sum(1, keepdims=True)
        runs = orc.runs(T, off, lens)
        N = sum(b - a for a, b in runs)
        for b, (lo, hi) in enumerate(runs):
            if hi > lo:
                total += 0.7 * (hi - lo) / N * (E * counts[b] / (K * (hi - lo)) * p[lo:hi].mean(0)).sum()
        return total

    got = orc.router_backward(logits, idx, K, norm, 2.5, dw, counts, 0.7, off, lens).dlogits
    for _ in range(20):
        d = rng.normal(size=logits.shape)
        slope = (loss(logits + 1e-6 * d) - loss(logits - 1e-6 * d)) / 2e-6
        assert abs((got * d).sum() - slope) <= 1e-8 * max(1.0, abs(slope))


def test_oracle_balance_of_an_even_load_is_the_coefficient():
    E, K = 64, 4
    logits = np.zeros((32, E))
    idx = (np.arange(32)[:, None] * K + np.arange(K)) % E
    b = orc.balance_loss(logits, idx, K, 0.3)
    assert abs(b.loss - 0.3) < 1e-15 and (b.counts == 2).all()
