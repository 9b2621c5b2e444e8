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


# ---- what a call may be given ------------------------------------------------------------------------

def test_no_tokens():
    """T = 0: zeros, and with accumulation what lay there."""
    cfg = config(64, 4)
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    counts, probs, loss = torch.full((2, 64), 7, dtype=I32, device="cuda"), torch.full((2, 64), 7.0, device="cuda"), z(1) + 7
    off = torch.tensor([0, 0, 0], dtype=I32).cuda()
    moe.moe_balance_loss(cfg, 0, z(0, 64), z(0, 4, dtype=I32), 1.0, counts, probs, loss, workspace(cfg, 0, 2), seq_offsets=off)
    assert not counts.any() and not probs.any() and loss.item() == 0
    for acc, want in ((False, 0.0), (True, 3.0)):
        drw = torch.full((64, 128), 3.0, device="cuda")
        moe.moe_router_backward(cfg, 0, z(0, 64), z(0, 4, dtype=I32), dtopk_w=z(0, 4), x=z(0, 128, dtype=BF), router_w=z(64, 128),
                                drouter_w=drw, accumulate_w=acc, dx=z(0, 128), ws=workspace(cfg, 0))
        assert (drw == want).all()


@pytest.mark.parametrize("T,E,H", [(50, 64, 128), (700, 128, 384)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")], ids=str)
def test_padding_may_hold_anything(T, E, H, bad):
    g = gen(8)
    K, cfg = 4, config(E, 4, H)
    off, lens = [0, T // 2, T], [T // 2 - 7, T - T // 2 - 3]
    pad = torch.ones(T, dtype=torch.bool)
    for o, n in zip(off, lens):
        pad[o:o + n] = False
    x, rw, logits, idx, dw, _, _, _, _ = backward_case(g, T, E, K, H, "one")
    idx[pad] = -1
    results = []
    for fill in (0.0, bad):
        x[pad], logits[pad], dw[pad] = fill, fill, fill
        o, n = on_gpu(off, lens)
        counts, probs = torch.empty(2, E, dtype=I32, device="cuda"), torch.empty(2, E, device="cuda")
        loss, drw = torch.empty(1, device="cuda"), torch.empty(E, H, device="cuda")
        dl, dx, ws = torch.empty(T, E, device="cuda"), torch.empty(T, H, device="cuda"), workspace(cfg, T, 2)
        moe.moe_balance_loss(cfg, T, logits.cuda(), idx.cuda(), 0.5, counts, probs, loss, ws, seq_offsets=o, seq_lens=n)
        moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), dtopk_w=dw.cuda(), counts=counts, coef=0.5, seq_offsets=o, seq_lens=n,
                                dlogits=dl, x=x.cuda(), router_w=rw.cuda(), drouter_w=drw, dx=dx, ws=ws)
        results.append((counts, probs, loss, dl, drw, dx))
        assert not dl[pad.cuda()].any() and not dx[pad.cuda()].any()
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=str)
def test_nonfinite_token_shows_and_stays(bad):
    g = gen(9)
    T, E, K, H = 100, 128, 4, 256
    cfg = config(E, K, H)
    x, rw, logits, idx, dw, counts, _, _, _ = backward_case(g, T, E, K, H, "one")
    dw[33, 1] = bad
    dl, drw, dx = torch.empty(T, E, device="cuda"), torch.empty(E, H, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")
    moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), dtopk_w=dw.cuda(), dlogits=dl, x=x.cuda(), router_w=rw.cuda(),
                            drouter_w=drw, dx=dx, ws=workspace(cfg, T))
    rest = torch.arange(T) != 33
    assert not torch.isfinite(dl[33]).all() and not torch.isfinite(dx[33]).any() and not torch.isfinite(drw).all()
    assert torch.isfinite(dl[rest.cuda()]).all() and torch.isfinite(dx[rest.cuda()]).all()
    logits[33] = bad
    probs, loss, counts = torch.empty(1, E, device="cuda"), torch.empty(1, device="cuda"), torch.empty(1, E, dtype=I32, device="cuda")
    moe.moe_balance_loss(cfg, T, logits.cuda(), idx.cuda(), 1.0, counts, probs, loss, workspace(cfg, T))
    assert np.isnan(loss.item()) == np.isnan(bad)   # an infinite logit is a score of one


def test_zero_and_one_scores():
    """Logits far out: scores of zero (a token of zeros counts as zeros) and of one."""
    T, E, K = 40, 64, 4
    cfg = config(E, K)
    logits = torch.full((T, E), 60.0)
    logits[:10] = -300.0
    logits[10:20] = -float("inf")
    logits[20:30, ::2] = -60.0
    idx = torch.arange(K, dtype=I32).repeat(T, 1)
    counts, probs, loss = torch.empty(1, E, dtype=I32, device="cuda"), torch.empty(1, E, device="cuda"), torch.empty(1, device="cuda")
    moe.moe_balance_loss(cfg, T, logits.cuda(), idx.cuda(), 1.0, counts, probs, loss, workspace(cfg, T))
    # (float64's sigmoid of -300 is no zero, fp32's is)
    want = orc.balance_loss(np.where(f64(logits) < -200, -np.inf, f64(logits)), idx.numpy(), K, 1.0)
    assert np.allclose(f64(probs), want.probs, rtol=1e-5, atol=1e-30) and abs(loss.item() - want.loss) <= 1e-5 * want.loss
    dl = torch.empty(T, E, device="cuda")
    moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), dtopk_w=torch.ones(T, K, device="cuda"), counts=counts, coef=1.0, dlogits=dl)
    assert torch.isfinite(dl).all() and not dl[:20].any()


@pytest.mark.parametrize("raw", [[-5, 3, 20, 2000], [0, 0, 60, 60], [-2**31, -1, 0, 61], [70, 80, 90, 2**31 - 1]], ids=str)
def test_sequence_offsets_are_clamped(raw):
    g = gen(10)
    T, E, K = 60, 64, 4
    cfg = config(E, K)
    logits, idx, lens = torch.randn(T, E, generator=g), ids(g, T, E, K), [5, -7, 2**31 - 1]
    counts, probs, loss = torch.empty(3, E, dtype=I32, device="cuda"), torch.empty(3, E, device="cuda"), torch.empty(1, device="cuda")
    dl = torch.empty(T, E, device="cuda")
    for n in (None, lens):
        o, m = on_gpu(raw, n)
        moe.moe_balance_loss(cfg, T, logits.cuda(), idx.cuda(), 1.0, counts, probs, loss, workspace(cfg, T, 3), seq_offsets=o, seq_lens=m)
        want = orc.balance_loss(f64(logits), idx.numpy(), K, 1.0, raw, n)
        assert np.array_equal(counts.cpu().numpy(), want.counts) and abs(loss.item() - want.loss) <= 1e-5 * want.loss
        moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), counts=counts, coef=1.0, seq_offsets=o, seq_lens=m, dlogits=dl)
        check_dlogits(dl, orc.router_backward(f64(logits), idx.numpy(), K, 1, 2.5, None, want.counts, 1.0, raw, n))


@pytest.mark.parametrize("T,B", [(300, 5000), (2, 3000), (40000, 65536)])
def test_many_sequences(T, B):
    g = gen(11)
    E, K = 64, 2
    cfg = config(E, K)
    off = torch.sort(torch.randint(0, T + 1, (B + 1,), generator=g))[0].tolist()
    logits, idx = torch.randn(T, E, generator=g), ids(g, T, E, K)
    counts, probs, loss = torch.empty(B, E, dtype=I32, device="cuda"), torch.empty(B, E, device="cuda"), torch.empty(1, device="cuda")
    o, _ = on_gpu(off, None)
    moe.moe_balance_loss(cfg, T, logits.cuda(), idx.cuda(), 2.0, counts, probs, loss, workspace(cfg, T, B), seq_offsets=o)
    want = orc.balance_loss(f64(logits), idx.numpy(), K, 2.0, off)
    assert np.array_equal(counts.cpu().numpy(), want.counts)
    assert np.all(np.abs(f64(probs) - want.probs) <= 1e-5 * want.probs) and abs(loss.item() - want.loss) <= 1e-5 * want.loss
    dl = torch.empty(T, E, device="cuda")
    moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), counts=counts, coef=2.0, seq_offsets=o, dlogits=dl)
    check_dlogits(dl, orc.router_backward(f64(logits), idx.numpy(), K, 1, 2.5, None, want.counts, 2.0, off))


@pytest.mark.parametrize("B", [1, 2, 63, 64, 65])
@pytest.mark.parametrize("T", [200, 3000, 20000])
@pytest.mark.parametrize("padded", [False, True])
def test_sequences_about_a_wave_of_them(T, B, padded):
    g = gen(12)
    E, K = 64, 2
    cfg = config(E, K)
    off = torch.sort(torch.randint(0, T + 1, (B + 1,), generator=g))[0].tolist()  # padding at both ends
    lens = [int(torch.randint(0, b - a + 1, (1,), generator=g)) for a, b in zip(off, off[1:])] if padded else None
    logits, idx, dw = torch.randn(T, E, generator=g), ids(g, T, E, K), torch.randn(T, K, generator=g)
    counts, probs, loss = torch.empty(B, E, dtype=I32, device="cuda"), torch.empty(B, E, device="cuda"), torch.empty(1, device="cuda")
    o, n = on_gpu(off, lens)
    moe.moe_balance_loss(cfg, T, logits.cuda(), idx.cuda(), 2.0, counts, probs, loss, workspace(cfg, T, B), seq_offsets=o, seq_lens=n)
    want = orc.balance_loss(f64(logits), idx.numpy(), K, 2.0, off, lens)
    assert np.array_equal(counts.cpu().numpy(), want.counts)
    rel = 2 * SCORE + (E / 64 + 8) * U32 + 264 * U32  # (as in test_balance_loss)
    assert np.all(np.abs(f64(probs) - want.probs) <= rel * want.probs + 1e-37)
    assert abs(loss.item() - want.loss) <= (rel + 4 * U32) * abs(want.loss)
    dl = torch.empty(T, E, device="cuda")
    moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), dtopk_w=dw.cuda(), counts=counts, coef=2.0, seq_offsets=o, seq_lens=n,
                            dlogits=dl)
    check_dlogits(dl, orc.router_backward(f64(logits), idx.numpy(), K, 1, 2.5, f64(dw), want.counts, 2.0, off, lens))


@pytest.mark.parametrize("E", [64, 512, 1024])
@pytest.mark.parametrize("T,B", [(40, 4), (65, 16), (500, 33), (5000, 300), (20000, 66)])
def test_short_and_long_sequences_together(T, B, E):
    g = gen(13)
    K = 4
    cfg = config(E, K)
    short = torch.arange(B) * (T // (3 * B))  # the last takes two thirds of the tokens
    off = [*short.tolist(), T]
    lens = [max(b - a - i % 3, 0) for i, (a, b) in enumerate(zip(off, off[1:]))]
    logits, idx = torch.randn(T, E, generator=g), ids(g, T, E, K)
    o, n = on_gpu(off, lens)
    want = orc.balance_loss(f64(logits), idx.numpy(), K, 2.0, off, lens)
    rel = 2 * SCORE + (E / 64 + 8) * U32 + 264 * U32  # (as in test_balance_loss)
    losses = []
    for _ in range(3):  # the parts, whichever workgroup ends last, in one order
        counts, probs, loss = torch.empty(B, E, dtype=I32, device="cuda"), torch.empty(B, E, device="cuda"), torch.empty(1, device="cuda")
        moe.moe_balance_loss(cfg, T, logits.cuda(), idx.cuda(), 2.0, counts, probs, loss, workspace(cfg, T, B), seq_offsets=o, seq_lens=n)
        assert np.array_equal(counts.cpu().numpy(), want.counts)
        assert np.all(np.abs(f64(probs) - want.probs) <= rel * want.probs + 1e-37)
        assert abs(loss.item() - want.loss) <= (rel + 4 * U32) * abs(want.loss)
        losses.append(loss.item())
    assert losses[0] == losses[1] == losses[2]


@pytest.mark.parametrize("size", [1e-36, 1e-20, 1e-6, 1e6, 1e20, 1e30], ids=str)
def test_gradients_of_any_size(size):
    """Scaled pieces: gradients, weights and columns of weights far from one, rows that span 2^30."""
    g = gen(12)
    T, E, K, H = 130, 128, 8, 256
    cfg = config(E, K, H, norm=0)
    x, rw, logits, idx, dw, _, _, _, _ = backward_case(g, T, E, K, H, "one")
    dw *= size * 2.0 ** torch.randint(-15, 16, (T, K), generator=g)
    rw *= 2.0 ** torch.randint(-20, 5, (1, H), generator=g)
    rw *= 2.0 ** torch.randint(-10, 1, (E, 1), generator=g)
    dl, drw, dx = torch.empty(T, E, device="cuda"), torch.empty(E, H, device="cuda"), torch.empty(T, H, device="cuda")
    moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), dtopk_w=dw.cuda(), dlogits=dl, x=x.cuda(), router_w=rw.cuda(),
                            drouter_w=drw, dx=dx, ws=workspace(cfg, T))
    d, w, xn = f64(dl), f64(rw), f64(x)
    want = d @ w
    # pieces of 2^-22, or of 2^-39 of a row's (column's) largest; results below fp32's normal range round to 2^-149
    low = 2.0 ** -38 * (np.abs(d).max(1)[:, None] * np.abs(w).sum(0) + np.abs(d).sum(1)[:, None] * np.abs(w).max(0))
    lim = (3 * 2.0 ** -22 + 6 * E * U32) * (np.abs(d) @ np.abs(w)) + low + U32 * np.abs(want) + 1e-44
    assert np.all(np.abs(f64(dx) - want) <= lim), np.max(np.abs(f64(dx) - want) / lim)
    # (a piece below fp32's normal range may be taken as zero by the matrix units: 2^-126 each)
    want, lim = d.T @ xn, 6 * T * U32 * (np.abs(d).T @ np.abs(xn)) + 3 * 2.0 ** -126 * np.abs(xn).sum(0) + 1e-37
    assert np.all(np.abs(f64(drw) - want) <= lim), np.max(np.abs(f64(drw) - want) / lim)


SHAPES = [(2100, 64, 384), (2500, 512, 640), (513, 1024, 1280), (4100, 128, 896), (9000, 64, 128), (64, 512, 2560), (8192, 512, 2560)]


@pytest.mark.parametrize("T,E,H", SHAPES, ids=str)
@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
def test_products_of_every_tile(T, E, H, f32):
    """Both tile sizes, reductions in one part and in many, sizes that fill no tile, against 64 bits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(13)
    K, cfg = 8, config(E, 8, H)
    x = torch.randn(T, H, generator=g, device="cuda").to(BF)
    rw = torch.randn(E, H, generator=g, device="cuda") * H ** -0.5
    logits = x.float() @ rw.t()
    idx = logits.topk(K, dim=1).indices.sort(dim=1).values.to(I32)
    dw = torch.randn(T, K, generator=g, device="cuda")
    dl, ws = torch.empty(T, E, device="cuda"), workspace(cfg, T)
    counts = torch.bincount(idx.reshape(-1).long(), minlength=E).view(1, E).to(I32)
    for which in ("both", "w", "x"):
        drw, dx = torch.full((E, H), 5.0, device="cuda"), torch.full((T, H), 2.0, dtype=F32 if f32 else BF, device="cuda")
        moe.moe_router_backward(cfg, T, logits, idx, dtopk_w=dw, counts=counts, coef=3.0, dlogits=dl, x=x, router_w=rw,
                                drouter_w=None if which == "x" else drw, accumulate_w=f32, dx=None if which == "w" else dx,
                                accumulate_x=f32, ws=ws.fill_(255))
        d = dl.double()
        if which != "x":
            want = d.t().contiguous() @ x.double() + (5.0 if f32 else 0.0)
            lim = 6 * T * U32 * (d.abs().t().contiguous() @ x.double().abs()) + 2 * U32 * (want.abs() + 5.0)
            assert ((drw.double() - want).abs() <= lim).all()
            # over 2^20 and more results the errors add as if by chance
            assert (drw.double() - want).norm() <= 1e-6 * want.norm()
        if which != "w":
            want = d @ rw.double() + (2.0 if f32 else 0.0)
            lim = (3 * 2.0 ** -22 if f32 else 2.01 * 2.0 ** -11) + 6 * E * U32
            lim = lim * (d.abs() @ rw.double().abs()) + (2 * U32 if f32 else HALF_BF16) * (want.abs() + 2.0)
            assert ((dx.double() - want).abs() <= lim).all()
            assert (dx.double() - want).norm() <= (1e-6 if f32 else 2.0 ** -9) * want.norm()


def test_large_batch_past_four_gibibytes():
    """Logits, planes and tokens of more than 4 GiB: sampled rows, the weight gradient against torch's in pieces."""
    T, E, H, K = 1_200_007, 1024, 128, 4
    cfg = config(E, K, H)
    g = torch.Generator(device="cuda")
    g.manual_seed(14)
    x, rw = torch.randn(T, H, generator=g, device="cuda").to(BF), torch.randn(E, H, generator=g, device="cuda")
    logits = torch.randn(T, E, generator=g, device="cuda")
    idx = torch.randint(0, E // K, (T, K), generator=g, device="cuda").to(I32) + torch.arange(K, device="cuda", dtype=I32) * (E // K)
    dw = torch.randn(T, K, generator=g, device="cuda")
    off = torch.tensor([0, 700_001, T], dtype=I32).cuda()
    counts, probs, loss = torch.empty(2, E, dtype=I32, device="cuda"), torch.empty(2, E, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(moe.moe_router_workspace_size(cfg, T, 2), dtype=torch.uint8, device="cuda")
    moe.moe_balance_loss(cfg, T, logits, idx, 1.0, counts, probs, loss, ws, seq_offsets=off)
    for b, (lo, hi) in enumerate(((0, 700_001), (700_001, T))):
        assert torch.equal(counts[b].long(), torch.bincount(idx[lo:hi].reshape(-1).long(), minlength=E))
        p = torch.zeros(E, dtype=torch.float64, device="cuda")
        for i in range(lo, hi, 100_000):
            s = torch.sigmoid(logits[i:min(i + 100_000, hi)].double())
            p += (s / s.sum(1, keepdim=True)).sum(0)
        assert ((probs[b].double() - p / (hi - lo)).abs() <= 1e-5 * p / (hi - lo)).all()
    dl, drw, dx = torch.empty(T, E, device="cuda"), torch.empty(E, H, device="cuda"), torch.empty(T, H, device="cuda")
    moe.moe_router_backward(cfg, T, logits, idx, dtopk_w=dw, counts=counts, coef=50.0, seq_offsets=off, dlogits=dl, x=x, router_w=rw,
                            drouter_w=drw, dx=dx, ws=ws)
    pick = torch.cat([torch.arange(50), torch.arange(700_000, 700_003), torch.arange(T - 50, T)])
    full = orc.router_backward(f64(logits[pick]), idx[pick].cpu().numpy(), K, 1, 2.5, f64(dw[pick]))
    f = counts.cpu().numpy() * E / (K * np.array([[700_001], [T - 700_001]]))
    s = 1 / (1 + np.exp(-f64(logits[pick])))
    p, fr = s / s.sum(1, keepdims=True), f[(pick.numpy() >= 700_001).astype(int)]
    bal = 50.0 / T * (fr - (fr * p).sum(1, keepdims=True)) * p * (1 - s)
    mag = full.dlogits_mag + 50.0 / T * (fr + (fr * p).sum(1, keepdims=True)) * p
    assert np.all(np.abs(f64(dl[pick]) - full.dlogits - bal) <= (4 * SCORE + 68 * U32) * mag + 1e-37)
    want = dl[pick].double() @ rw.double()
    assert (dx[pick].double() - want).norm() <= 1e-6 * want.norm()
    want = torch.zeros(E, H, dtype=torch.float64, device="cuda")
    for i in range(0, T, 100_000):
        want += dl[i:i + 100_000].double().t().contiguous() @ x[i:i + 100_000].double()
    # 16 parts or more of a reduction over 1.2 million tokens, sums of at most 40,000 terms in fp32
    assert (drw.double() - want).norm() <= 2e-5 * want.norm()


# ---- as they are used ----------------------------------------------------------------------------------

class RouterStep:
    """The router's part of training steps: routing, loss, backward, norm of two gradients, the clipped step."""

    def __init__(self, seed, T=200, E=128, K=4, H=256):
        g = gen(seed)
        self.cfg, self.T = config(E, K, H), T
        self.x, self.rw = torch.randn(T, H, generator=g).to(BF).cuda(), (torch.randn(E, H, generator=g) * H ** -0.5).cuda()
        self.dw, self.other = torch.randn(T, K, generator=g).cuda(), torch.randn(50_001, generator=g).to(BF).cuda()
        e = lambda *s, **k: torch.empty(*s, device="cuda", **k)  # noqa: E731
        self.idx, self.w, self.logits = e(T, K, dtype=I32), e(T, K), e(T, E)
        self.off = torch.tensor([0, T // 3, T], dtype=I32).cuda()
        self.counts, self.probs, self.loss = e(2, E, dtype=I32), e(2, E), e(1)
        self.drw, self.dx, self.norm, self.coef = e(E, H), e(T, H, dtype=BF), e(1), e(1)
        self.m, self.v = torch.zeros(E, H, device="cuda"), torch.zeros(E, H, device="cuda")
        self.clipped = [torch.empty(E, H, dtype=BF, device="cuda"), torch.empty(50_001, device="cuda")]
        self.ws = torch.empty(max(moe.moe_workspace_size(self.cfg, T), moe.moe_router_workspace_size(self.cfg, T, 2)),
                              dtype=torch.uint8, device="cuda")
        self.plan = moe.MoEGradPlan([self.drw, self.other], out=self.clipped)
        self.nws = torch.empty(self.plan.workspace_size, dtype=torch.uint8, device="cuda")
        self.adam = moe.MoEAdamWPlan([self.rw], [self.drw], [self.m], [self.v], weight_decay=0.01)
        self.step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def run(self):
        moe.moe_route_logits(self.cfg, self.T, self.x, self.rw, None, self.idx, self.w, self.logits, self.ws)
        moe.moe_balance_loss(self.cfg, self.T, self.logits, self.idx, 0.1, self.counts, self.probs, self.loss, self.ws, seq_offsets=self.off)
        moe.moe_router_backward(self.cfg, self.T, self.logits, self.idx, dtopk_w=self.dw, counts=self.counts, coef=0.1,
                                seq_offsets=self.off, x=self.x, router_w=self.rw, drouter_w=self.drw, dx=self.dx, ws=self.ws)
        moe.moe_grad_norm(self.plan, 1.0, self.norm, self.coef, self.nws)
        moe.moe_grad_clip(self.plan, self.coef)
        self.step.add_(1)
        moe.moe_adamw_step(self.adam, lr=1e-2, step=self.step, grad_scale=self.coef)

    def results(self):
        return [self.idx, self.w, self.logits, self.counts, self.probs, self.loss, self.drw, self.dx, self.norm, self.coef,
                *self.clipped, self.rw, self.m, self.v]


def test_router_steps_are_deterministic_and_clipped():
    a, b = RouterStep(20), RouterStep(20)
    for _ in range(3):
        a.run()
        b.run()
        assert all(torch.equal(x, y) for x, y in zip(a.results(), b.results()))
    want = np.sqrt((f64(a.drw) ** 2).sum() + (f64(a.other) ** 2).sum())
    assert abs(a.norm.item() - want) <= 20 * U32 * want and abs(a.coef.item() - 1 / want) <= 20 * U32 / want
    total = np.sqrt(sum((f64(t) ** 2).sum() for t in a.clipped))
    assert abs(total - 1.0) <= HALF_BF16


def test_router_steps_in_a_graph():
    """A captured step replayed several times, with eager work between, against the same steps run eagerly."""
    a, b, eager = RouterStep(21), RouterStep(21), RouterStep(22, T=77)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        eager.run()                        # warm up, on other buffers
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run()
    for _ in range(4):
        graph.replay()
        eager.run()
        b.run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.results(), b.results()))


def test_router_steps_on_two_streams():
    solo = [RouterStep(s, T=900) for s in (23, 24)]
    for s in solo:
        s.run()
    torch.cuda.synchronize()
    both, streams = [RouterStep(s, T=900) for s in (23, 24)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(1):
        for s, st in zip(both, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s, t in zip(solo, both):
        assert all(torch.equal(x, y) for x, y in zip(s.results(), t.results()))


def test_router_steps_from_two_host_threads():
    import threading
    solo = [RouterStep(s, T=500) for s in (25, 26)]
    both = [RouterStep(s, T=500) for s in (25, 26)]
    for s in solo:
        s.run()
    torch.cuda.synchronize()
    failed = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                s.run()
        except Exception as e:  # pragma: no cover
            failed.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in both]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for s, t in zip(solo, both):
        assert all(torch.equal(x, y) for x, y in zip(s.results(), t.results()))


def test_layer_with_its_router_against_autograd():
    """A layer's whole backward pass: experts, router and balance loss, against float64 autograd.  On the way to
    any result at most six roundings to bf16 follow each other, each at most 2^-8 of its value; the 2-norm of a
    result may be off by twice their sum.  (Routing weights and their gradient are fp32, the router's own
    operators lose less than 2^-16.)"""
    g = gen(27)
    T, E, K, H, I, coef = 60, 64, 4, 128, 128, 5.0
    cfg = config(E, K, H)
    with_rows = config(E, K, H)
    with_rows.num_shared_experts = 1       # the combine then adds the rows behind the routed ones
    P = T * K
    x, rw = torch.randn(T, H, generator=g).to(BF).cuda(), (torch.randn(E, H, generator=g) * H ** -0.5).cuda()
    gate, up = [(torch.randn(E, I, H, generator=g) * H ** -0.5).to(BF).cuda() for _ in range(2)]
    down = (torch.randn(E, H, I, generator=g) * I ** -0.5).to(BF).cuda()
    dout = torch.randn(T, H, generator=g).to(BF).cuda()
    e = lambda *s, **k: torch.empty(*s, device="cuda", **k)  # noqa: E731
    ws = e(max(moe.moe_workspace_size(cfg, T), moe.moe_router_workspace_size(cfg, T)), dtype=torch.uint8)
    idx, w, logits = e(T, K, dtype=I32), e(T, K), e(T, E)
    n, off, tok, inv = e(E + 1, dtype=I32), e(E + 2, dtype=I32), e(P, dtype=I32), e(T, K, dtype=I32)
    moe.moe_route_logits(cfg, T, x, rw, None, idx, w, logits, ws)
    moe.moe_dispatch(cfg, T, idx, n, off, tok, inv, ws)
    o, pos, ones = off[:E + 1], inv.view(-1), torch.ones(T, K, device="cuda")
    gm, um, hm, y, out = e(P, I, dtype=BF), e(P, I, dtype=BF), e(P, I, dtype=BF), e(P, H), e(T, H, dtype=BF)
    moe.moe_grouped_gemm(x, gate, o, gm, row_map=tok)
    moe.moe_grouped_gemm(x, up, o, um, row_map=tok)
    moe.moe_swiglu(gm, um, hm, row_w=w.view(-1), pos=pos)
    moe.moe_grouped_gemm(hm, down, o, y)
    moe.moe_combine(cfg, T, y, inv, ones, out)
    counts, probs, loss = e(1, E, dtype=I32), e(1, E), e(1)
    moe.moe_balance_loss(cfg, T, logits, idx, coef, counts, probs, loss, ws)
    # backward
    dh, dg, du, dw = e(P, I, dtype=BF), e(P, I, dtype=BF), e(P, I, dtype=BF), e(T, K)
    rows, dx, drw = e(P + T, H), e(T, H, dtype=BF), e(E, H)
    d_gate, d_up, d_down = e(E, I, H), e(E, I, H), e(E, H, I)
    moe.moe_grouped_gemm_dgrad(dout, down, o, dh, row_map=tok)
    moe.moe_grouped_gemm_wgrad(dout, hm, o, d_down, dy_map=tok)
    moe.moe_swiglu_backward(gm, um, dh, dg, du, row_w=w.view(-1), pos=pos, drow_w=dw.view(-1))
    moe.moe_grouped_gemm_dgrad(dg, gate, o, rows[:P], dy2=du, w2=up)
    moe.moe_grouped_gemm_wgrad(dg, x, o, d_gate, x_map=tok)
    moe.moe_grouped_gemm_wgrad(du, x, o, d_up, x_map=tok)
    moe.moe_router_backward(cfg, T, logits, idx, dtopk_w=dw, counts=counts, coef=coef, x=x, router_w=rw, drouter_w=drw, dx=rows[P:], ws=ws)
    moe.moe_combine(with_rows, T, rows, inv, ones, dx)

    leaves = [t.double().cpu().requires_grad_() for t in (x, rw, gate, up, down)]
    xd, rd, gd, ud, dd = leaves
    ix = idx.long().cpu()
    s = torch.sigmoid(xd @ rd.t())
    sk = s.gather(1, ix)
    wt = 2.5 * sk / sk.sum(1, keepdim=True)
    ref = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            ex = int(ix[t, k])
            ref[t] = ref[t] + wt[t, k] * (dd[ex] @ (torch.nn.functional.silu(gd[ex] @ xd[t]) * (ud[ex] @ xd[t])))
    bal = (torch.bincount(ix.reshape(-1), minlength=E) * E / (K * T) * (s / s.sum(1, keepdim=True)).mean(0)).sum() * coef
    ((ref * dout.double().cpu()).sum() + bal).backward()
    bound = 2 * 6 * HALF_BF16
    assert abs(loss.item() - bal.item()) <= 1e-5 * bal.item()
    assert np.linalg.norm(f64(out) - ref.detach().numpy()) <= bound * np.linalg.norm(ref.detach().numpy())
    for got, leaf in zip((dx, drw, d_gate, d_up, d_down), leaves):
        want = leaf.grad.numpy()
        assert np.linalg.norm(f64(got) - want) <= bound * np.linalg.norm(want)
    # the gradients' norm, and a step of the router weight with it
    grads = [d_gate, d_up, d_down, drw]
    norm, coef_t = e(1), e(1)
    plan = moe.MoEGradPlan(grads)
    moe.moe_grad_norm(plan, 0.5, norm, coef_t, e(plan.workspace_size, dtype=torch.uint8))
    want = np.sqrt(sum((f64(t) ** 2).sum() for t in grads))
    assert abs(norm.item() - want) <= 20 * U32 * want
    states = [[torch.zeros_like(rw) for _ in range(2)] for _ in range(2)]
    params = [rw.clone(), rw.clone()]
    moe.moe_adamw_step(moe.MoEAdamWPlan([params[0]], [drw], [states[0][0]], [states[0][1]]), lr=1e-2, step=1, grad_scale=coef_t)
    moe.moe_grad_clip(plan, coef_t)        # in place
    moe.moe_adamw_step(moe.MoEAdamWPlan([params[1]], [drw], [states[1][0]], [states[1][1]]), lr=1e-2, step=1)
    assert torch.equal(params[0], params[1]) and torch.equal(states[0][0], states[1][0])


# ---- the gradients' plan --------------------------------------------------------------------------------

def test_wrong_gradient_image_writes_nothing():
    t = torch.ones(20000, device="cuda")
    plan = moe.MoEGradPlan([t])
    other = moe.MoEGradPlan([torch.ones(100, device="cuda"), torch.ones(100, device="cuda"), torch.ones(100, device="cuda")])
    norm, coef, ws = torch.full((1,), 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda"), torch.empty(plan.workspace_size, dtype=torch.uint8, device="cuda")
    for image in (torch.zeros_like(plan.image), other.image):
        plan.at = image.data_ptr()
        moe.moe_grad_norm(plan, 1.0, norm, coef, ws)
        moe.moe_grad_clip(plan, coef)
        assert norm.item() == 7 and coef.item() == 7 and (t == 1).all()


def test_clipping_by_one_leaves_the_bits():
    t = torch.tensor([1.0, -0.0, float("nan"), float("inf"), 1e-45], device="cuda")
    before = t.view(torch.int32).clone()
    moe.moe_grad_clip(moe.MoEGradPlan([t]), torch.ones(1, device="cuda"))
    assert torch.equal(t.view(torch.int32), before)


def test_no_gradients():
    empty = [torch.empty(0, device="cuda"), torch.empty(0, dtype=BF, device="cuda")]
    plan = moe.MoEGradPlan(empty)
    norm, coef = torch.full((1,), 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda")
    moe.moe_grad_norm(plan, 0.0, norm, coef, torch.empty(plan.workspace_size, dtype=torch.uint8, device="cuda"), scale=0.5)
    moe.moe_grad_clip(plan, coef)
    assert norm.item() == 0 and coef.item() == 0.5


def test_gradient_past_two_to_the_32_values():
    n = 2 ** 32 + 2 ** 14 + 3
    t = torch.full((n,), 0.5, dtype=BF, device="cuda")
    t[-1] = 4096.0
    plan = moe.MoEGradPlan([t])
    norm, coef = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    moe.moe_grad_norm(plan, 1024.0, norm, coef, torch.empty(plan.workspace_size, dtype=torch.uint8, device="cuda"))
    want = np.sqrt(0.25 * (n - 1) + 2.0 ** 24)
    assert abs(norm.item() - want) <= 20 * U32 * want
    moe.moe_grad_clip(plan, torch.tensor([0.5], device="cuda"))
    assert t[-1].item() == 2048 and t[0].item() == 0.25 and (t[2 ** 32 - 5:2 ** 32 + 5] == 0.25).all()


def test_gradient_table_outlives_a_plan_that_is_dropped():
    """The table's memory is kept until work on another stream has run (its address is not handed out again)."""
    t = torch.ones(300_000, device="cuda")
    plan = moe.MoEGradPlan([t])
    size, address = plan.image.numel(), plan.image.data_ptr()
    norm, ws = torch.empty(1, device="cuda"), torch.empty(plan.workspace_size, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
        moe.moe_grad_norm(plan, 1.0, norm, None, ws)
    del plan
    again = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(a.data_ptr() != address for a in again)
    torch.cuda.synchronize()
    assert abs(norm.item() - np.sqrt(300_000)) < 1e-2


# ---- at the ends of the range ----------------------------------------------------------------------------

@pytest.mark.parametrize("T,E,H", [(1, 64, 128), (64, 512, 2560), (1333, 128, 640), (700, 1024, 256), (2500, 512, 640)], ids=str)
def test_bf16_dx_is_rounded_once(T, E, H):
    """dx in bf16 is the fp32 result rounded to bf16, also where a sum cancels: beside that rounding it may be off by
    what dx in fp32 may be (operands in two fp16 pieces, sums in fp32), not by a share of the magnitudes summed."""
    g = gen(30)
    K, cfg = 8, config(E, 8, H)
    x, rw, logits, idx, dw, counts, _, _, _ = backward_case(g, T, E, K, H, "one")
    dl, dx, dx32 = torch.empty(T, E, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, device="cuda")
    for out in (dx, dx32):
        moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), dtopk_w=dw.cuda(), counts=counts.cuda(), coef=3.0, dlogits=dl,
                                router_w=rw.cuda(), dx=out, ws=workspace(cfg, T))
    d, w = f64(dl), f64(rw)
    want = d @ w
    own = (3 * 2.0 ** -22 + 6 * E * U32) * (np.abs(d) @ np.abs(w))
    lim = own + HALF_BF16 * (np.abs(want) + own) + 1e-37
    err = np.abs(f64(dx) - want)
    assert np.all(err <= lim), f"err/tol {np.max(err / lim):.1f}, {np.mean(err > lim):.2%} of the values"
    assert torch.equal(dx, dx32.to(BF))


@pytest.mark.parametrize("max_norm", [0.0, 1.0, float("inf")])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf")], ids=str)
def test_infinite_gradient_has_a_coefficient_of_zero(bad, max_norm):
    grads = [torch.ones(100000, device="cuda"), torch.ones(9, dtype=BF, device="cuda")]
    grads[1][3] = bad
    plan = moe.MoEGradPlan(grads)
    norm, coef = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(plan.workspace_size, dtype=torch.uint8, device="cuda")
    moe.moe_grad_norm(plan, max_norm, norm, coef, ws, scale=0.5)
    assert np.isposinf(norm.item()) and coef.item() == 0


@pytest.mark.parametrize("centre", [-60.0, -86.0, -88.0, -95.0, -103.0, -120.0])
@pytest.mark.parametrize("E,K", [(64, 4), (512, 8), (1024, 16)])
@pytest.mark.parametrize("T", [40, 700])
def test_tokens_of_tiny_scores(T, E, K, centre):
    """Shares are quotients of scores: they do not depend on whether fp32 holds the scores themselves (nor a large
    gradient times a score's reciprocal).  Every third token is an ordinary one."""
    g = gen(31)
    cfg = config(E, K)
    logits, idx, dw = torch.randn(T, E, generator=g) * 2, ids(g, T, E, K), torch.randn(T, K, generator=g)
    logits[torch.arange(T) % 3 > 0] += centre
    off, lens = sequences("padded", T)
    B = len(off) - 1
    o, n = on_gpu(off, lens)
    counts, probs, loss = torch.empty(B, E, dtype=I32, device="cuda"), torch.empty(B, E, device="cuda"), torch.empty(1, device="cuda")
    moe.moe_balance_loss(cfg, T, logits.cuda(), idx.cuda(), 0.25, counts, probs, loss, workspace(cfg, T, B), seq_offsets=o, seq_lens=n)
    want = orc.balance_loss(f64(logits), idx.numpy(), K, 0.25, off, lens)
    assert np.array_equal(counts.cpu().numpy(), want.counts)
    rel = 2 * SCORE + (E / 64 + 8) * U32 + 264 * U32  # (as in test_balance_loss)
    assert np.all(np.abs(f64(probs) - want.probs) <= rel * want.probs + 1e-37)
    assert abs(loss.item() - want.loss) <= (rel + 4 * U32) * abs(want.loss)
    dl = torch.empty(T, E, device="cuda")
    scale = torch.tensor([65536.0], device="cuda")
    for mix in (None, dw):
        moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), dtopk_w=None if mix is None else mix.cuda(), counts=counts, coef=10.0,
                                dloss=scale, seq_offsets=o, seq_lens=n, dlogits=dl)
        check_dlogits(dl, orc.router_backward(f64(logits), idx.numpy(), K, 1, 2.5, None if mix is None else f64(mix), want.counts,
                                              10.0 * 65536.0, off, lens))


def test_no_tokens_leave_the_bits_of_a_gradient_added_to():
    cfg = config(64, 4)
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    drw = z(64, 128)
    drw[::2] = -0.0
    before = drw.view(I32).clone()
    moe.moe_router_backward(cfg, 0, z(0, 64), z(0, 4, dtype=I32), dtopk_w=z(0, 4), x=z(0, 128, dtype=BF), router_w=z(64, 128),
                            drouter_w=drw, accumulate_w=True, dx=z(0, 128), ws=workspace(cfg, 0))
    assert torch.equal(drw.view(I32), before)


@pytest.mark.parametrize("norm", [0, 1])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")], ids=str)
def test_logits_that_are_not_finite(bad, norm):
    """A NaN shows where the token's gradient depends on it: at a chosen expert, with a balance loss at any.  An infinity
    is a score of one or zero like any other and shows nowhere."""
    g = gen(32)
    T, E, K, H = 70, 64, 4, 128
    cfg = config(E, K, H, norm=norm)
    x, rw, clean, idx, dw, counts, _, _, _ = backward_case(g, T, E, K, H, "one")
    chosen, other = int(idx[33, 1]), int(next(e for e in range(E) if e not in idx[33].tolist()))
    for e in (chosen, other):
        logits = clean.clone()
        logits[33, e] = bad
        for mix, balance in ((True, False), (False, True), (True, True)):
            dl, drw, dx = torch.empty(T, E, device="cuda"), torch.empty(E, H, device="cuda"), torch.empty(T, H, device="cuda")
            moe.moe_router_backward(cfg, T, logits.cuda(), idx.cuda(), dtopk_w=dw.cuda() if mix else None,
                                    counts=counts.cuda() if balance else None, coef=0.5, dlogits=dl, x=x.cuda(), router_w=rw.cuda(),
                                    drouter_w=drw, dx=dx, ws=workspace(cfg, T))
            shows = np.isnan(bad) and (balance or e == chosen)
            assert bool(torch.isfinite(dl[33]).all()) != shows and bool(torch.isfinite(drw).all()) != shows
            assert bool(torch.isfinite(dx[33]).all()) != shows
            rest = (torch.arange(T) != 33).cuda()
            assert torch.isfinite(dl[rest]).all() and torch.isfinite(dx[rest]).all()
            if not np.isnan(bad):
                want = orc.router_backward(f64(logits), idx.numpy(), K, norm, 2.5, f64(dw) if mix else None,
                                           counts.numpy() if balance else None, 0.5, None, None)
                check_dlogits(dl, want)
