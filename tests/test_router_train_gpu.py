"""The operators that train the router, and the gradient norm with clipping, on the GPU against their
float64 definitions.

Tolerances.  A score is a sigmoid in fp32: the power of two, the reciprocal and five roundings around
them are each at most one unit in the last place, so a score and its complement are off by at most
SCORE = 8 of 2^-23 of themselves.  A sum of n terms is off by n 2^-24 times the sum of their magnitudes in any
order.  One rounding to bf16 adds 2^-8 of the value, to fp32 2^-24.
"""
import numpy as np
import pytest
import torch

import sparse_moe_layer_bailingmoev3_amd as moe
from oracle import router_oracle as orc

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
HALF_BF16 = 2.0 ** -8
U32 = 2.0 ** -24
SCORE = 8 * 2.0 ** -23


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def f64(t):
    return t.detach().double().cpu().numpy()


def config(E, K, H=128, G=8, norm=1, scale=2.5, TG=4):
    return moe.MoEConfig(hidden_size=H, num_experts=E, num_experts_per_tok=K, n_group=G, topk_group=TG, moe_intermediate_size=128,
                         num_shared_experts=0, shared_intermediate_size=128, norm_topk_prob=norm, routed_scaling_factor=scale,
                         swiglu_limit=0.0, shared_swiglu_limit=0.0, expert_weight_format=0, expert_act_format=0)


def workspace(cfg, T, B=1):
    """Filled with NaN patterns: nothing may be read that the call did not write."""
    return torch.full((moe.moe_router_workspace_size(cfg, T, B),), 255, dtype=torch.uint8, device="cuda")


def ids(g, T, E, K):
    return torch.rand(T, E, generator=g).topk(K, dim=1).indices.sort(dim=1).values.to(I32)


# (offsets, lens) of T tokens
def sequences(kind, T):
    if kind == "one":
        return None, None
    if kind == "padded_one":
        return None, [max(T - 3, 0)]
    if kind == "ragged":  # gaps on both sides, empty runs
        a, b, c = T // 7, T // 3, 2 * T // 3
        return [a, b, b, b, c, max(T - 1, c)], None
    if kind == "padded":
        a, b = T // 3, T // 2
        return [0, a, b, b, T], [a // 2, b - a, 5, max(T - b - 1, 0)]
    if kind == "single_tokens":
        return list(range(T + 1)), None
    assert kind == "none"
    return [0, T], [0]


KINDS = ["one", "padded_one", "ragged", "padded", "single_tokens", "none"]


def on_gpu(off, lens):
    t = lambda v: None if v is None else torch.tensor(v, dtype=I32).cuda()  # noqa: E731
    return t(off), t(lens)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 2, 31, 97, 700])
@pytest.mark.parametrize("E,K", [(64, 1), (128, 4), (512, 8), (1024, 16)])
def test_balance_loss(E, K, T, kind):
    g = gen(1)
    cfg = config(E, K)
    logits, idx = torch.randn(T, E, generator=g) * 2, ids(g, T, E, K)
    idx[:: 5, 0] = -1
    idx[1:: 7, K - 1] = E
    off, lens = sequences(kind, T)
    B = 1 if off is None else len(off) - 1
    counts, probs = torch.empty(B, E, dtype=I32, device="cuda"), torch.empty(B, E, device="cuda")
    loss = torch.empty(1, device="cuda")
    o, n = on_gpu(off, lens)
    moe.moe_balance_loss(cfg, T, logits.cuda(), idx.cuda(), 0.25, counts, probs, loss, workspace(cfg, T, B), seq_offsets=o, seq_lens=n)
    want = orc.balance_loss(f64(logits), idx.numpy(), K, 0.25, off, lens)
    assert np.array_equal(counts.cpu().numpy(), want.counts)
    # a share is a score over a sum of E scores; its mean adds up to 256 shares in fp32, the rest in 64 bits
    rel = 2 * SCORE + (E / 64 + 8) * U32 + 264 * U32
    assert np.all(np.abs(f64(probs) - want.probs) <= rel * want.probs + 1e-37)
    assert abs(loss.item() - want.loss) <= (rel + 4 * U32) * abs(want.loss)


def test_balance_counts_are_the_dispatch_counts():
    g = gen(2)
    T, E, K = 300, 128, 4
    cfg = config(E, K)
    idx = ids(g, T, E, K).cuda()
    counts, probs, loss = torch.empty(1, E, dtype=I32, device="cuda"), torch.empty(1, E, device="cuda"), torch.empty(1, device="cuda")
    moe.moe_balance_loss(cfg, T, torch.zeros(T, E, device="cuda"), idx, 1.0, counts, probs, loss, workspace(cfg, T))
    n, off = torch.empty(E + 1, dtype=I32, device="cuda"), torch.empty(E + 2, dtype=I32, device="cuda")
    tok, inv = torch.empty(T * K, dtype=I32, device="cuda"), torch.empty(T * K, dtype=I32, device="cuda")
    ws = torch.empty(moe.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    moe.moe_dispatch(cfg, T, idx, n, off, tok, inv, ws)
    assert torch.equal(n[:E], counts[0])
    assert abs(loss.item() - 1.0) <= 1e-5  # even scores: every share is 1 / E, so any load gives coef


def backward_case(g, T, E, K, H, kind):
    off, lens = sequences(kind, T)
    B = 1 if off is None else len(off) - 1
    x, rw = torch.randn(T, H, generator=g).to(BF), torch.randn(E, H, generator=g) * H ** -0.5
    logits, idx = torch.randn(T, E, generator=g) * 2, ids(g, T, E, K)
    dw = torch.randn(T, K, generator=g)
    counts = torch.from_numpy(orc.balance_loss(f64(logits), idx.numpy(), K, 1.0, off, lens).counts)
    return x, rw, logits, idx, dw, counts, off, lens, B


def check_dlogits(got, want):
    # two scores, the chosen ones' sum (16), the sum over a sequence's share (2 E / 64 + 8 terms), six operations
    tol = (4 * SCORE + (16 + 40 + 12) * U32) * want.dlogits_mag + 1e-37
    err = np.abs(f64(got) - want.dlogits)
    assert np.all(err <= tol), f"err/tol {np.max(err / tol):.2f} at {np.unravel_index(np.argmax(err / tol), err.shape)}"
    return tol


def check_products(want, tol, x, rw, dw=None, dx=None, dw0=None, dx0=None):
    """The products' own roundings (drouter_w: none, three exact pieces; dx: operands in two fp16 pieces,
    2^-22 each, and what is left out as much again, or, for a result in bf16, in one, 2^-11 each at half a
    step; sums in fp32) and the logits' gradient's."""
    xn, wn = np.abs(f64(x)), np.abs(f64(rw))
    d = np.abs(want.dlogits)
    T, E = d.shape
    if dw is not None:
        old = 0 if dw0 is None else f64(dw0)
        ref = want.dlogits.T @ f64(x) + old
        lim = tol.T @ xn + 2 * 3 * T * U32 * (d.T @ xn) + U32 * (np.abs(ref) + np.abs(old)) + 1e-37
        err = np.abs(f64(dw) - ref)
        assert np.all(err <= lim), f"drouter_w: err/tol {np.max(err / lim):.2f}"
    if dx is not None:
        old = 0 if dx0 is None else f64(dx0)
        ref = want.dlogits @ f64(rw) + old
        piece = 2.01 * 2.0 ** -11 if dx.dtype is BF else 3 * 2.0 ** -22
        lim = tol @ wn + (piece + 2 * 3 * E * U32) * (d @ wn) + (HALF_BF16 if dx.dtype is BF else U32) * np.abs(ref) + U32 * np.abs(old) + 1e-37
        err = np.abs(f64(dx) - ref)
        assert np.all(err <= lim), f"dx: err/tol {np.max(err / lim):.2f}"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,E,K,H", [(1, 64, 1, 128), (2, 128, 4, 384), (31, 64, 8, 128), (65, 512, 8, 256), (300, 128, 2, 640),
                                     (97, 1024, 16, 128), (1333, 64, 4, 256)], ids=str)
@pytest.mark.parametrize("norm", [0, 1])
def test_backward(T, E, K, H, kind, norm):
    g = gen(3)
    cfg = config(E, K, H, norm=norm)
    x, rw, logits, idx, dw, counts, off, lens, B = backward_case(g, T, E, K, H, kind)
    idx[2:: 5, 0] = -1
    o, n = on_gpu(off, lens)
    dloss = torch.tensor([0.75]).cuda()
    args = dict(counts=counts.cuda(), coef=0.5, dloss=dloss, seq_offsets=o, seq_lens=n, x=x.cuda(), router_w=rw.cuda())
    dl, drw = torch.empty(T, E, device="cuda"), torch.randn(E, H, generator=g).cuda()
    dx = torch.randn(T, H, generator=g).cuda()
    drw0, dx0 = drw.clone(), dx.clone()
    ws = workspace(cfg, T, B)
    moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), dtopk_w=dw.cuda(), dlogits=dl, drouter_w=drw, accumulate_w=True, dx=dx,
                            accumulate_x=True, ws=ws, **args)
    want = orc.router_backward(f64(logits), idx.numpy(), K, norm, 2.5, f64(dw), counts.numpy(), 0.5 * 0.75, off, lens)
    tol = check_dlogits(dl, want)
    check_products(want, tol, x, rw, drw, dx, drw0, dx0)
    # without the gradient of the mixing weights, written anew, dx in bf16
    drw, dxb = torch.full((E, H), float("nan"), device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")
    moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), drouter_w=drw, dx=dxb, ws=ws.fill_(255), **args)
    want = orc.router_backward(f64(logits), idx.numpy(), K, norm, 2.5, None, counts.numpy(), 0.5 * 0.75, off, lens)
    tol = (4 * SCORE + 68 * U32) * want.dlogits_mag + 1e-37
    check_products(want, tol, x, rw, drw, dxb)
    # the mixing weights alone
    moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), dtopk_w=dw.cuda(), dlogits=dl)
    check_dlogits(dl, orc.router_backward(f64(logits), idx.numpy(), K, norm, 2.5, f64(dw), None, 0.0, off, lens))


def test_backward_against_autograd_and_differences():
    g = gen(4)
    T, E, K, H = 40, 64, 4, 128
    cfg = config(E, K, H)
    off, lens = [0, 11, 30, 40], [11, 15, 10]
    x, rw = torch.randn(T, H, generator=g).to(BF), torch.randn(E, H, generator=g) * H ** -0.5
    leaves = [x.double().requires_grad_(), rw.double().requires_grad_()]
    idx = (leaves[0] @ leaves[1].t()).topk(K, dim=1).indices.sort(dim=1).values
    dw = torch.randn(T, K, generator=g).double()

    def loss_of(x, rw):
        s = torch.sigmoid(x @ rw.t())
        sk = s.gather(1, idx)
        w = 2.5 * sk / sk.sum(1, keepdim=True)
        p = s / s.sum(1, keepdim=True)
        N, bal = sum(lens), 0.0
        for b, n in enumerate(lens):
            r = slice(off[b], off[b] + n)
            f = torch.bincount(idx[r].reshape(-1), minlength=E) * E / (K * n)
            bal = bal + n / N * (f * p[r].mean(0)).sum()
        return (w * dw).sum() + 3.0 * bal

    loss_of(*leaves).backward()
    logits = (leaves[0] @ leaves[1].t()).detach().float()
    o, n = on_gpu(off, lens)
    counts, probs, loss = torch.empty(3, E, dtype=I32, device="cuda"), torch.empty(3, E, device="cuda"), torch.empty(1, device="cuda")
    ws = workspace(cfg, T, 3)
    moe.moe_balance_loss(cfg, T, logits.cuda(), idx.to(I32).cuda(), 3.0, counts, probs, loss, ws, seq_offsets=o, seq_lens=n)
    drw, dx = torch.empty(E, H, device="cuda"), torch.empty(T, H, device="cuda")
    moe.moe_router_backward(cfg, T, logits.cuda(), idx.to(I32).cuda(), dtopk_w=dw.float().cuda(), counts=counts, coef=3.0, seq_offsets=o,
                            seq_lens=n, x=x.cuda(), router_w=rw.cuda(), drouter_w=drw, dx=dx, ws=ws)
    for got, leaf in zip((dx, drw), leaves):
        want = leaf.grad.numpy()
        # logits of up to 4 rounded to fp32 move a score by 2^-22; the rest as in the other tests
        bound = 2.0 ** -16
        assert np.linalg.norm(f64(got) - want) <= bound * np.linalg.norm(want)
        d = torch.randn(leaf.shape, generator=g, dtype=torch.float64)
        e = 1e-6
        with torch.no_grad():
            moved = [loss_of(*[l + sgn * e * d if l is leaf else l for l in leaves]) for sgn in (1, -1)]
        slope = float(moved[0] - moved[1]) / (2 * e)
        dot = float((f64(got) * d.numpy()).sum())
        assert abs(dot - slope) <= bound * np.linalg.norm(want) * np.linalg.norm(d.numpy()) + 1e-7 * abs(slope)


@pytest.mark.parametrize("T", [1, 5, 64, 257, 1000, 4100])
@pytest.mark.parametrize("E,H", [(64, 128), (512, 2560)])
def test_route_logits(T, E, H):
    g = gen(5)
    K = 8
    cfg = config(E, K, H)
    x, rw = torch.randn(T, H, generator=g).to(BF).cuda(), (torch.randn(E, H, generator=g) * H ** -0.5).cuda()
    bias = (torch.randn(E, generator=g) * 0.1).cuda()
    ws = torch.empty(moe.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    a, b = [(torch.empty(T, K, dtype=I32, device="cuda"), torch.empty(T, K, device="cuda")) for _ in range(2)]
    logits = torch.empty(T, E, device="cuda")
    moe.moe_route(cfg, T, x, rw, bias, *a, ws)
    moe.moe_route_logits(cfg, T, x, rw, bias, *b, logits, ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    want, mag = f64(x) @ f64(rw).T, np.abs(f64(x)) @ np.abs(f64(rw)).T
    assert np.all(np.abs(f64(logits) - want) <= 2 * H * U32 * mag)


# ---- norm and clipping -----------------------------------------------------------------------------

SIZES = [1, 7, 8, 2047, 2048, 16384, 16385, 100003, 0, 33]


@pytest.mark.parametrize("out", [None, BF, F32], ids=["in_place", "to_bf16", "to_fp32"])
@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9, float("inf")])
@pytest.mark.parametrize("scale", [1.0, 0.125, -3.0])
def test_grad_norm_and_clip(out, max_norm, scale):
    g = gen(6)
    grads = [(torch.randn(n, generator=g) * 0.01).to(BF if i % 3 else F32).cuda() for i, n in enumerate(SIZES)]
    before = [f64(t) for t in grads]
    outs = None if out is None else [torch.full((n,), float("nan"), dtype=out, device="cuda") for n in SIZES]
    plan = moe.MoEGradPlan(grads, out=outs)
    norm, coef = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.full((plan.workspace_size,), 255, dtype=torch.uint8, device="cuda")
    moe.moe_grad_norm(plan, max_norm, norm, coef, ws, scale=scale)
    want = abs(scale) * np.sqrt(sum((t ** 2).sum() for t in before))
    wcoef = scale * (1.0 if want <= max_norm else max_norm / want)
    # 32 squares and sums of a lane in fp32, halved by the root
    assert abs(norm.item() - want) <= 20 * U32 * want and abs(coef.item() - wcoef) <= 20 * U32 * abs(wcoef)
    moe.moe_grad_clip(plan, coef)
    c = float(coef.item())
    for t, b in zip(grads if out is None else outs, before):
        assert np.all(np.abs(f64(t) - b * c) <= (HALF_BF16 * 1.01 if t.dtype is BF else U32) * np.abs(b * c) + 1e-40)
    if out is not None:
        assert all(np.array_equal(f64(t), b) for t, b in zip(grads, before))


@pytest.mark.parametrize("size", [1e-38, 1e-25, 1e-15, 1e15, 1e18, 1e25, 1e37], ids=str)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_grad_norm_of_very_small_and_large_gradients(size, dtype):
    g = gen(7)
    grads = [(torch.randn(n, generator=g) * size).clamp(-3e38, 3e38).to(dtype).cuda() for n in (5, 20000)]
    if size == 1e15:
        grads.append((torch.randn(3000, generator=g) * 1e-30).to(dtype).cuda())
    plan = moe.MoEGradPlan(grads)
    norm = torch.empty(1, device="cuda")
    moe.moe_grad_norm(plan, 1.0, norm, None, torch.empty(plan.workspace_size, dtype=torch.uint8, device="cuda"), scale=1 / 64)
    want = np.sqrt(sum((f64(t) ** 2).sum() for t in grads)) / 64
    assert abs(norm.item() - want) <= 20 * U32 * want + 2.0 ** -149


@pytest.mark.parametrize("bad,norm_is,coef_is", [(float("nan"), np.isnan, np.isnan), (float("inf"), np.isposinf, lambda v: v == 0),
                                                 (-float("inf"), np.isposinf, lambda v: v == 0)], ids=["nan", "inf", "-inf"])
def test_grad_norm_not_finite(bad, norm_is, coef_is):
    grads = [torch.ones(100000, device="cuda"), torch.ones(9, dtype=BF, device="cuda")]
    grads[0][77777] = bad
    plan = moe.MoEGradPlan(grads)
    norm, coef = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    moe.moe_grad_norm(plan, 1.0, norm, coef, torch.empty(plan.workspace_size, dtype=torch.uint8, device="cuda"))
    assert norm_is(norm.item()) and coef_is(coef.item())
