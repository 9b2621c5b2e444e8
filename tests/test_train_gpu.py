"""The operators that train a layer's experts on the GPU, against their float64 definitions.

Tolerances.  A product summed in fp32 over n terms is off by at most n 2^-24 times the sum of the
terms' magnitudes whatever the order (every addition rounds by at most 2^-24 of a partial sum that
these bound; the matrix instruction's own inner sums are counted twice over by taking 2n), and one
rounding to bf16 adds 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import sparse_moe_layer_bailingmoev3_amd as moe
from oracle import train_oracle as orc

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF_BF16 = 2.0 ** -8
U32 = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def offsets_of(counts, first=0):
    return torch.tensor([first] + list(first + np.cumsum(counts)), dtype=torch.int32).cuda()


def check(got, want, mag, n, bf16):
    tol = 2 * n * U32 * mag + (HALF_BF16 * np.abs(want) if bf16 else U32 * np.abs(want)) + 1e-37
    err = np.abs(f64(got) - want)
    bad = err > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}, err/tol {np.max(err / tol):.2f}"


COUNTS = {
    "one_row": [1],
    "one_row_of_many": [0, 0, 1, 0],
    "ragged": [3, 0, 17, 1, 64, 0, 5],
    "long": [300, 1, 0, 129],
    "tiles": [128, 256, 127],
    "empty": [0, 0, 0],
}
DIMS = [(128, 128), (136, 264), (8, 8), (768, 72), (40, 520)]


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("kind", ["bf16", "fp32", "acc", "mapped"])
def test_forward(counts, dims, kind):
    g = gen(1)
    c, (N, K) = COUNTS[counts], dims
    first, tail = 2, 3            # rows of no group on both sides
    off, P = offsets_of(c, first), first + sum(c) + tail
    T = 11 if kind == "mapped" else P
    x, w = randn(g, T, K), randn(g, len(c), N, K)
    m = torch.randint(-1, T + 1, (P,), generator=g, dtype=torch.int32).cuda() if kind == "mapped" else None
    y = randn(g, P, N, dtype=BF if kind in ("bf16", "mapped") else F32)
    before = f64(y)
    moe.moe_grouped_gemm(x, w, off, y, row_map=m, accumulate=kind == "acc")
    want, mag = orc.grouped_forward(f64(x), f64(w), off.cpu().numpy(), before, None if m is None else m.cpu().numpy(), kind == "acc")
    check(y, want, mag, K, y.dtype == BF)
    assert np.array_equal(f64(y)[:first], before[:first]) and np.array_equal(f64(y)[P - tail:], before[P - tail:])


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("kind", ["bf16", "pair", "acc_pair", "mapped"])
def test_dgrad(counts, dims, kind):
    g = gen(2)
    c, (N, K) = COUNTS[counts], dims
    first, tail = 1, 2
    off, P = offsets_of(c, first), first + sum(c) + tail
    T = 9 if kind == "mapped" else P
    pair = "pair" in kind
    dy, w = randn(g, T, N), randn(g, len(c), N, K)
    dy2, w2 = (randn(g, T, N), randn(g, len(c), N, K)) if pair else (None, None)
    m = torch.randint(-1, T + 1, (P,), generator=g, dtype=torch.int32).cuda() if kind == "mapped" else None
    dx = randn(g, P, K, dtype=F32 if pair else BF)
    before = f64(dx)
    moe.moe_grouped_gemm_dgrad(dy, w, off, dx, row_map=m, dy2=dy2, w2=w2, accumulate=kind == "acc_pair")
    want, mag = orc.grouped_dgrad(f64(dy), f64(w), off.cpu().numpy(), before, None if m is None else m.cpu().numpy(),
                                  f64(dy2) if pair else None, f64(w2) if pair else None, kind == "acc_pair")
    check(dx, want, mag, 2 * N, dx.dtype == BF)
    assert np.array_equal(f64(dx)[:first], before[:first]) and np.array_equal(f64(dx)[P - tail:], before[P - tail:])


@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("kind", ["bf16", "fp32", "acc", "mapped_x", "mapped_both"])
def test_wgrad(counts, dims, kind):
    g = gen(3)
    c, (N, K) = COUNTS[counts], dims
    first, tail = 1, 2
    off, P = offsets_of(c, first), first + sum(c) + tail
    T = 13
    mx = torch.randint(-1, T + 1, (P,), generator=g, dtype=torch.int32).cuda() if kind.startswith("mapped") else None
    md = torch.randint(-1, T + 1, (P,), generator=g, dtype=torch.int32).cuda() if kind == "mapped_both" else None
    dy, x = randn(g, T if md is not None else P, N), randn(g, T if mx is not None else P, K)
    dw = randn(g, len(c), N, K, dtype=F32 if kind in ("fp32", "acc") else BF)
    before = f64(dw)
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw, dy_map=md, x_map=mx, accumulate=kind == "acc")
    num = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    want, mag = orc.grouped_wgrad(f64(dy), f64(x), off.cpu().numpy(), before, num(md), num(mx), kind == "acc")
    check(dw, want, mag, max(c) + 1, dw.dtype == BF)


def test_grouped_strided_operands():
    """Operands and results that are columns of wider buffers."""
    g = gen(4)
    c, N, K = [5, 130, 0, 33], 72, 136
    off, P = offsets_of(c), sum(c)
    wide, w = randn(g, P, K + N + 24), randn(g, len(c), N, K)
    x, dy = wide[:, 8:8 + K], wide[:, 16 + K:16 + K + N]
    ybuf = torch.zeros(P, N + 40, dtype=F32, device="cuda")
    y = ybuf[:, 16:16 + N]
    moe.moe_grouped_gemm(x, w, off, y)
    o = off.cpu().numpy()
    want, mag = orc.grouped_forward(f64(x), f64(w), o, np.zeros((P, N)))
    check(y, want, mag, K, False)
    assert not ybuf[:, :16].any() and not ybuf[:, 16 + N:].any()
    dxbuf = torch.zeros(P, K + 8, dtype=BF, device="cuda")
    moe.moe_grouped_gemm_dgrad(dy, w, off, dxbuf[:, :K])
    want, mag = orc.grouped_dgrad(f64(dy), f64(w), o, np.zeros((P, K)))
    check(dxbuf[:, :K], want, mag, N, True)
    assert not dxbuf[:, K:].any()
    dw = torch.empty(len(c), N, K, dtype=F32, device="cuda")
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw)
    want, mag = orc.grouped_wgrad(f64(dy), f64(x), o, np.zeros(dw.shape))
    check(dw, want, mag, max(c), False)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_grouped_nonfinite_stays_where_it_is(bad):
    """Values outside a group, its rows and its columns never reach a sum."""
    g = gen(5)
    c, N, K = [3, 5, 0, 70], 40, 72
    off, P = offsets_of(c, 4), 4 + sum(c) + 4
    x, w, dy = randn(g, P + 8, K), randn(g, len(c), N, K), randn(g, P + 8, N)
    o = off.cpu().numpy()
    for t in (x, dy):                     # rows of no group, and the rows behind the matrix
        t[:4] = bad
        t[P - 4:] = bad
    w[2] = bad                            # the empty group's weights
    x, dy = x[:P], dy[:P]
    y = torch.zeros(P, N, dtype=F32, device="cuda")
    dx = torch.zeros(P, K, dtype=F32, device="cuda")
    dw = torch.zeros(len(c), N, K, dtype=F32, device="cuda")
    moe.moe_grouped_gemm(x, w, off, y)
    moe.moe_grouped_gemm_dgrad(dy, w, off, dx)
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw)
    assert torch.isfinite(y).all() and torch.isfinite(dx).all() and torch.isfinite(dw).all()
    assert not dw[2].any()
    x[5] = bad                            # one row of group 0: its own results only
    moe.moe_grouped_gemm(x, w, off, y)
    fin = torch.isfinite(y).all(1)
    assert not fin[5] and fin[:5].all() and fin[6:].all()
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw)
    assert not torch.isfinite(dw[0]).any() and torch.isfinite(dw[1:]).all()
    assert o[0] == 4


def test_wgrad_skipped_row_may_hold_anything():
    """A position without a row in one operand does not count, whatever the other holds there."""
    g = gen(6)
    off = offsets_of([6])
    dy, x = randn(g, 4, 16), randn(g, 6, 24)
    md = torch.tensor([0, -1, 2, 4, 3, 1], dtype=torch.int32).cuda()
    x[1] = float("nan")
    x[3] = float("inf")
    dw = torch.empty(1, 16, 24, dtype=F32, device="cuda")
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw, dy_map=md)
    keep = [0, 2, 4, 5]
    want = f64(dy)[md.cpu().numpy()[keep]].T @ f64(x)[keep]
    assert np.allclose(f64(dw)[0], want, rtol=1e-5, atol=1e-5)


# ---- SwiGLU --------------------------------------------------------------------------------------

def swiglu_inputs(g, R, C, n, skip):
    gate, up, dh = randn(g, R, C, scale=3.0), randn(g, R, C, scale=2.0), randn(g, R, C)
    pos = torch.randperm(R, generator=g)[:n].to(torch.int32)
    if skip:
        pos[::3] = -1
        pos[1::7] = R
    return gate, up, dh, pos.cuda(), (torch.rand(n, generator=g) + 0.1).cuda()


@pytest.mark.parametrize("cols", [8, 136, 768, 1032])
@pytest.mark.parametrize("rows,n,skip", [(1, 1, False), (37, 37, False), (50, 30, True)])
@pytest.mark.parametrize("limit", [0.0, 4.0])
def test_swiglu(cols, rows, n, skip, limit):
    g = gen(7)
    gate, up, dh, pos, w = swiglu_inputs(g, rows, cols, n, skip)
    h = randn(g, rows, cols)
    dgate, dup = randn(g, rows, cols), randn(g, rows, cols)
    keep = [f64(t) for t in (h, dgate, dup)]
    drow = torch.full((n,), 7.0, device="cuda")
    moe.moe_swiglu(gate, up, h, limit=limit, row_w=w, pos=pos)
    moe.moe_swiglu_backward(gate, up, dh, dgate, dup, limit=limit, row_w=w, pos=pos, drow_w=drow)
    p = pos.cpu().numpy()
    ok = (p >= 0) & (p < rows)
    r = p[ok]
    G, U, DH, W = f64(gate)[r], f64(up)[r], f64(dh)[r], f64(w)[ok]
    sig, _, free, s = orc.swiglu(G, U, limit)
    # the fp32 sigmoid: exp of an argument rounded by |g| 2^-24, and three more operations
    rel = (np.abs(G) + 8) * 2 * U32
    want = s * W[:, None]
    assert (np.abs(f64(h)[r] - want) <= HALF_BF16 * np.abs(want) * (1 + 2 * HALF_BF16) + 4 * rel * np.abs(want) + 1e-37).all()
    dg, du, dw = orc.swiglu_backward(G, U, DH, limit, W)
    da = np.abs(DH * W[:, None] * U * sig)
    assert (np.abs(f64(dgate)[r] - dg) <= HALF_BF16 * np.abs(dg) * (1 + 2 * HALF_BF16) + 4 * rel * da * (1 + np.abs(G)) + 1e-37).all()
    assert (np.abs(f64(dup)[r] - du) <= HALF_BF16 * np.abs(du) * (1 + 2 * HALF_BF16) + 4 * rel * np.abs(du) + 1e-37).all()
    terms = np.abs(DH * s)
    assert (np.abs(f64(drow)[ok] - dw) <= (4 * rel * terms).sum(1) + cols * U32 * terms.sum(1) + 1e-37).all()
    assert (f64(drow)[~ok] == 0).all()
    rest = np.setdiff1d(np.arange(rows), r)
    for t, b in zip((h, dgate, dup), keep):
        assert np.array_equal(f64(t)[rest], b[rest])


def test_swiglu_plain_rows_and_packed_buffers():
    """No positions, no weights, gate and up side by side in one buffer; gradients likewise."""
    g = gen(8)
    R, C = 19, 40
    buf, dbuf = randn(g, R, 2 * C), torch.zeros(R, 2 * C, dtype=BF, device="cuda")
    dh, h = randn(g, R, C), torch.empty(R, C, dtype=BF, device="cuda")
    gate, up = buf[:, :C], buf[:, C:]
    moe.moe_swiglu(gate, up, h)
    moe.moe_swiglu_backward(gate, up, dh, dbuf[:, :C], dbuf[:, C:])
    _, _, _, s = orc.swiglu(f64(gate), f64(up), 0)
    dg, du, _ = orc.swiglu_backward(f64(gate), f64(up), f64(dh), 0, np.ones(R))
    assert np.allclose(f64(h), s, rtol=2.1 * HALF_BF16 / 2, atol=1e-6)
    assert np.allclose(f64(dbuf[:, :C]), dg, rtol=2.1 * HALF_BF16 / 2, atol=1e-5)
    assert np.allclose(f64(dbuf[:, C:]), du, rtol=2.1 * HALF_BF16 / 2, atol=1e-5)


def test_swiglu_extreme_values():
    """Saturated gates, infinities and NaN behave as the formula does; the clamp keeps NaN."""
    vals = torch.tensor([-100.0, -30.0, -0.0, 0.0, 30.0, 100.0, float("nan"), float("inf")], dtype=BF).cuda()
    gate, up = vals.repeat(8, 1), vals[:, None].expand(8, 8).contiguous()
    h = torch.empty(8, 8, dtype=BF, device="cuda")
    moe.moe_swiglu(gate, up, h, limit=5.0)
    a = torch.nn.functional.silu(gate.double()) * up.double()
    want = a.clamp(-5, 5).to(BF)
    assert torch.equal(torch.isnan(h), torch.isnan(want))
    fin = ~torch.isnan(want)
    assert torch.allclose(h[fin].double(), want[fin].double(), atol=1e-6, rtol=HALF_BF16)


def test_swiglu_backward_against_differences():
    """Gradients against central differences of the float64 forward, away from the clamp's border."""
    g = gen(9)
    R, C, L = 6, 24, 3.0
    gate, up, dh, pos, w = swiglu_inputs(g, R, C, R, False)
    dgate, dup = torch.empty_like(gate), torch.empty_like(gate)
    drow = torch.empty(R, device="cuda")
    moe.moe_swiglu_backward(gate, up, dh, dgate, dup, limit=L, row_w=w, pos=pos, drow_w=drow)
    p = pos.cpu().numpy()
    W = np.empty(R)
    W[p] = f64(w)
    G, U, DH = f64(gate), f64(up), f64(dh)
    f = lambda G, U, W: (DH * W[:, None] * orc.swiglu(G, U, L)[3])  # noqa: E731
    e = 1e-5
    a = np.abs(orc.swiglu(G, U, L)[1])
    far = np.abs(a - L) > 1e-3
    # a difference quotient is off by e^2 times the third derivative (below 10 |dh w u|) and by 1e-16 / e
    slack = 1e-6 * (1 + np.abs(DH * W[:, None]) * (1 + np.abs(U)) * (1 + np.abs(G)))
    ng = (f(G + e, U, W) - f(G - e, U, W)) / (2 * e)
    nu = (f(G, U + e, W) - f(G, U - e, W)) / (2 * e)
    nw = (f(G, U, W + e) - f(G, U, W - e)).sum(1) / (2 * e)
    assert (np.abs(f64(dgate) - ng) <= HALF_BF16 * 1.01 * np.abs(ng) + slack)[far].all()
    assert (np.abs(f64(dup) - nu) <= HALF_BF16 * 1.01 * np.abs(nu) + slack)[far].all()
    assert (np.abs(f64(drow) - nw[p]) <= 1e-4 * (1 + np.abs(nw[p]))).all()


# ---- AdamW ---------------------------------------------------------------------------------------

SIZES = [1, 7, 128, 129, 1000, 8192, 8193, 20000, 0]


def adamw_inputs(seed, pdt, gdt, eight, master, sizes=SIZES):
    g = gen(seed)
    params = [randn(g, n, dtype=pdt, scale=0.05) for n in sizes]
    grads = [randn(g, n, dtype=gdt, scale=1e-2) for n in sizes]
    ms = [p.float() + 1e-4 for p in params] if master else None
    if eight:
        m = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes]
        v = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes]
        sc = [torch.zeros(-(-n // 128), device="cuda") for n in sizes]
        sv = [torch.zeros(-(-n // 128), device="cuda") for n in sizes]
    else:
        m, v = [randn(g, n, dtype=F32, scale=1e-2) for n in sizes], [randn(g, n, dtype=F32, scale=1e-2).square() for n in sizes]
        sc = sv = None
    return params, grads, ms, m, v, sc, sv


@pytest.mark.parametrize("pdt,master", [(BF, False), (BF, True), (F32, False)], ids=["bf16", "bf16_master", "fp32"])
@pytest.mark.parametrize("gdt", [BF, F32], ids=["gbf16", "gfp32"])
@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
def test_adamw(pdt, master, gdt, eight):
    params, grads, ms, m, v, sc, sv = adamw_inputs(10, pdt, gdt, eight, master)
    wd = [0.1 * (i % 2) for i in range(len(SIZES))]
    plan = moe.MoEAdamWPlan(params, grads, m, v, master=ms, exp_avg_scale=sc, exp_avg_sq_scale=sv, weight_decay=wd)
    lr, betas, eps, seed = 1e-2, (0.9, 0.999), 1e-8, 77
    for step in (1, 2, 3):
        before = [f64(t) for t in (ms if master else params)]
        if eight:
            old = [(orc.state_decode(a.cpu().numpy(), s.cpu().numpy(), True), orc.state_decode(b.cpu().numpy(), q.cpu().numpy(), False))
                   for a, s, b, q in zip(m, sc, v, sv)]
        else:
            old = [(a.cpu().numpy(), b.cpu().numpy()) for a, b in zip(m, v)]
        moe.moe_adamw_step(plan, lr=lr, step=step, betas=betas, eps=eps, seed=seed)
        for i, n in enumerate(SIZES):
            wm, wv = orc.adamw_moments(old[i][0], old[i][1], grads[i].float().cpu().numpy(), betas)
            if eight:
                for codes, scales, x, signed in ((m[i], sc[i], wm, True), (v[i], sv[i], wv, False)):
                    wc, ws = orc.state_encode(x, signed, i, seed, step)
                    assert np.array_equal(scales.cpu().numpy(), ws)
                    assert np.array_equal(codes.cpu().numpy(), wc)
                    out = torch.empty(n, device="cuda")
                    moe.moe_adamw_dequantise(codes, scales, out, signed)
                    assert np.array_equal(out.cpu().numpy(), orc.state_decode(wc, ws, signed))
            else:  # the same fp32 operations: the same bits
                assert np.array_equal(m[i].cpu().numpy(), wm) and np.array_equal(v[i].cpu().numpy(), wv)
            want = orc.adamw_param(before[i], wm, wv, lr, step, betas, eps, wd[i])
            # about ten fp32 operations on the update and three on the parameter
            tol = 16 * U32 * (np.abs(want - before[i]) + lr) + 4 * U32 * np.abs(before[i])
            if master:
                assert (np.abs(f64(ms[i]) - want) <= tol).all()
                assert torch.equal(params[i], ms[i].to(BF))
            else:
                assert (np.abs(f64(params[i]) - want) <= tol + (HALF_BF16 * np.abs(want) if pdt == BF else 0)).all()


def test_adamw_device_scalars_match_host():
    """lr, step and the gradient scale from device memory: the same states bit for bit."""
    a, b = (adamw_inputs(11, BF, BF, True, True) for _ in range(2))
    mk = lambda t: moe.MoEAdamWPlan(t[0], t[1], t[3], t[4], master=t[2], exp_avg_scale=t[5], exp_avg_sq_scale=t[6])  # noqa: E731
    pa, pb = mk(a), mk(b)
    for g in b[1]:
        g.mul_(0.5)                       # exact
    moe.moe_adamw_step(pa, lr=torch.tensor([1e-3], device="cuda"), step=torch.tensor([5], device="cuda"), seed=3,
                       grad_scale=torch.tensor([0.5], device="cuda"))
    moe.moe_adamw_step(pb, lr=float(np.float32(1e-3)), step=5, seed=3)
    for i in (3, 4, 5, 6):
        for x, y in zip(a[i], b[i]):
            assert torch.equal(x, y)
    for x, y in zip(a[2], b[2]):
        assert torch.allclose(x, y, rtol=1e-6, atol=1e-9)


def test_adamw_nonfinite_gradient_shows():
    """An infinite or NaN gradient is not lost in the 8-bit states; other blocks keep their values."""
    for bad in (float("nan"), float("inf")):
        params, grads, _, m, v, sc, sv = adamw_inputs(12, BF, F32, True, False, [512])
        grads[0][130] = bad
        plan = moe.MoEAdamWPlan(params, grads, m, v, exp_avg_scale=sc, exp_avg_sq_scale=sv)
        moe.moe_adamw_step(plan, lr=1e-3, step=1)
        out = torch.empty(512, device="cuda")
        moe.moe_adamw_dequantise(m[0], sc[0], out, True)
        assert not torch.isfinite(out[128:256]).any() or not torch.isfinite(out[130])
        assert torch.isfinite(out[:128]).all() and torch.isfinite(out[256:]).all()


def test_adamw_rounding_is_unbiased():
    """A constant gradient: with rounding to nearest the second moment would stand still; the mean
    over many values follows the fp32 recurrence.  One rounding errs by at most an eighth of the
    value, independently from value to value and step to step, so the mean of n values after s
    steps is off by less than 5 (0.125 / sqrt(3)) sqrt(s (1-b2)^2 ...) / sqrt(n); 2 % leaves that far behind."""
    n, steps, betas = 128 * 512, 40, (0.9, 0.99)
    p, gr = [torch.zeros(n, device="cuda")], [torch.full((n,), 0.25, device="cuda")]
    gr[0][::2] = 1.0                      # half the values sit below the block's maximum
    m, v = ([torch.zeros(n, dtype=torch.uint8, device="cuda")] for _ in range(2))
    sc, sv = ([torch.zeros(n // 128, device="cuda")] for _ in range(2))
    plan = moe.MoEAdamWPlan(p, gr, m, v, exp_avg_scale=sc, exp_avg_sq_scale=sv)
    for s in range(1, steps + 1):
        moe.moe_adamw_step(plan, lr=0.0, step=s, betas=betas, seed=5)
    out = torch.empty(n, device="cuda")
    moe.moe_adamw_dequantise(v[0], sv[0], out, False)
    for start, g in ((0, 1.0), (1, 0.25)):
        want = g * g * (1 - betas[1] ** steps)
        assert abs(out[start::2].double().mean().item() / want - 1) < 0.02
    moe.moe_adamw_dequantise(m[0], sc[0], out, True)
    for start, g in ((0, 1.0), (1, 0.25)):
        want = g * (1 - betas[0] ** steps)
        assert abs(out[start::2].double().mean().item() / want - 1) < 0.02


# ---- offsets past 32 bits ------------------------------------------------------------------------

def test_grouped_operands_past_four_gibibytes():
    """Rows far apart in a buffer of more than 4 GiB, by position and through maps, in every product."""
    g = gen(20)
    R, LD, N, K = 1100, 1 << 21, 40, 72
    buf = torch.empty(R, LD, dtype=BF, device="cuda")        # 4.6 GB
    x, dy = buf[:, 8:8 + K], buf[:, 1024:1024 + N]
    x.copy_(randn(g, R, K))
    dy.copy_(randn(g, R, N))
    dy2 = buf[:, 4096:4096 + N]
    dy2.copy_(randn(g, R, N))
    counts = [500, 0, 350, 250]
    off, o = offsets_of(counts), offsets_of(counts).cpu().numpy()
    w, w2 = randn(g, 4, N, K), randn(g, 4, N, K)
    for mapped in (False, True):
        m = torch.randint(-1, R + 1, (R,), generator=g, dtype=torch.int32).cuda() if mapped else None
        mn = None if m is None else m.cpu().numpy()
        y, dx = torch.zeros(R, N, device="cuda"), torch.zeros(R, K, device="cuda")
        dw = torch.zeros(4, N, K, device="cuda")
        moe.moe_grouped_gemm(x, w, off, y, row_map=m)
        moe.moe_grouped_gemm_dgrad(dy, w, off, dx, row_map=m)
        moe.moe_grouped_gemm_wgrad(dy, x, off, dw, dy_map=m, x_map=m)
        X, DY, W = f64(x), f64(dy), f64(w)
        check(y, *orc.grouped_forward(X, W, o, np.zeros((R, N)), mn), K, False)
        check(dx, *orc.grouped_dgrad(DY, W, o, np.zeros((R, K)), mn), N, False)
        check(dw, *orc.grouped_wgrad(DY, X, o, np.zeros((4, N, K)), mn, mn), 500, False)
        moe.moe_grouped_gemm_dgrad(dy, w, off, dx, row_map=m, dy2=dy2, w2=w2)
        check(dx, *orc.grouped_dgrad(DY, W, o, np.zeros((R, K)), mn, f64(dy2), f64(w2)), 2 * N, False)


# ---- how the operators are called ----------------------------------------------------------------

def test_grouped_most_groups():
    """1025 groups (a full layer's experts and a shared one), most of them empty."""
    g = gen(21)
    counts = np.zeros(1025, int)
    counts[[0, 63, 64, 511, 512, 1023, 1024]] = [3, 1, 2, 17, 1, 1, 40]
    off, P, N, K = offsets_of(counts), int(counts.sum()), 24, 40
    x, w, dy = randn(g, P, K), randn(g, 1025, N, K), randn(g, P, N)
    o = off.cpu().numpy()
    y, dx = torch.zeros(P, N, device="cuda"), torch.zeros(P, K, device="cuda")
    dw = torch.full((1025, N, K), 5.0, device="cuda")
    moe.moe_grouped_gemm(x, w, off, y)
    moe.moe_grouped_gemm_dgrad(dy, w, off, dx)
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw)
    check(y, *orc.grouped_forward(f64(x), f64(w), o, np.zeros((P, N))), K, False)
    check(dx, *orc.grouped_dgrad(f64(dy), f64(w), o, np.zeros((P, K))), N, False)
    check(dw, *orc.grouped_wgrad(f64(dy), f64(x), o, np.zeros((1025, N, K))), 40, False)


# every tile shape that a size rule can take: (positions a group, groups, weights)
SHAPES = [(1, 70, (768, 136)), (4, 40, (768, 136)), (16, 64, (264, 520)), (40, 24, (520, 264)), (70, 130, (264, 136)),
          (200, 12, (264, 136)), (300, 70, (264, 520)), (900, 2, (264, 136)), (64, 1, (2560, 768)), (3000, 1, (136, 72)),
          (60, 130, (776, 776)), (150, 200, (72, 136)), (40, 60, (136, 776)), (90, 130, (520, 136)), (300, 60, (136, 264)),
          (20, 300, (520, 520)), (500, 100, (72, 136))]


@pytest.mark.parametrize("rows,G,dims", SHAPES, ids=str)
def test_grouped_tile_shapes(rows, G, dims):
    """Groups around an average size, whichever tile shape that picks; every group checked."""
    g = gen(22)
    N, K = dims
    counts = np.maximum(0, rows + torch.randint(-rows // 2, rows // 2 + 2, (G,), generator=g).numpy())
    off, P = offsets_of(counts), int(counts.sum())
    T = P // 2 + 1
    x, w, dy = randn(g, T, K), randn(g, G, N, K), randn(g, T, N)
    m = torch.randint(0, T, (P,), generator=g, dtype=torch.int32).cuda()
    o, mn = off.cpu().numpy(), m.cpu().numpy()
    y, dx = torch.zeros(P, N, device="cuda"), torch.zeros(P, K, dtype=BF, device="cuda")
    dw = torch.ones(G, N, K, device="cuda")
    moe.moe_grouped_gemm(x, w, off, y, row_map=m)
    moe.moe_grouped_gemm_dgrad(dy, w, off, dx, row_map=m)
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw, dy_map=m, x_map=m, accumulate=True)
    X, W, DY = f64(x), f64(w), f64(dy)
    check(y, *orc.grouped_forward(X, W, o, np.zeros((P, N)), mn), K, False)
    check(dx, *orc.grouped_dgrad(DY, W, o, np.zeros((P, K)), mn), N, True)
    check(dw, *orc.grouped_wgrad(DY, X, o, np.ones((G, N, K)), mn, mn, True), int(counts.max()) + 1, False)


def test_no_rows():
    off = offsets_of([0, 0])
    e = lambda n: torch.empty(0, n, dtype=BF, device="cuda")  # noqa: E731
    w = torch.ones(2, 16, 24, dtype=BF, device="cuda")
    moe.moe_grouped_gemm(e(24), w, off, e(16))
    moe.moe_grouped_gemm_dgrad(e(16), w, off, e(24))
    dw = torch.ones(2, 16, 24, device="cuda")
    moe.moe_grouped_gemm_wgrad(e(16), e(24), off, dw, accumulate=True)
    assert (dw == 1).all()
    moe.moe_grouped_gemm_wgrad(e(16), e(24), off, dw)
    assert not dw.any()
    y = torch.ones(3, 16, dtype=BF, device="cuda")           # positions whose rows do not exist
    moe.moe_grouped_gemm(e(24), w, offsets_of([1, 2]), y, row_map=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert not y.any()
    moe.moe_swiglu(e(8), e(8), e(8))
    drow = torch.ones(2, device="cuda")
    moe.moe_swiglu_backward(e(8), e(8), e(8), e(8), e(8), pos=torch.tensor([0, -1], dtype=torch.int32, device="cuda"), drow_w=drow)
    assert not drow.any()


def test_wrong_adamw_image_writes_nothing():
    """The device copy of another plan is recognised by the kernel."""
    mk = lambda n: moe.MoEAdamWPlan(*([torch.ones(n, device="cuda")] for _ in range(4)))  # noqa: E731
    a, b = mk(100), mk(20000)
    a.image, a.at = b.image, b.at
    moe.moe_adamw_step(a, lr=1.0, step=1)
    for p in (a, b):
        assert all((t[0] == 1).all() for t in p._keep.values())


class Step:
    """The operators of one training step of a small layer, on buffers of its own."""

    def __init__(self, seed, T=70, E=8, K=2, H=136, I=72, limit=3.0):
        g = gen(seed)
        self.T, self.K, self.E, self.limit = T, K, E, limit
        idx = torch.stack([torch.randperm(E, generator=g)[:K].sort().values for _ in range(T)])
        flat = idx.reshape(-1)
        order = torch.argsort(flat, stable=True)
        inv = torch.empty(T * K, dtype=torch.int32)
        inv[order] = torch.arange(T * K, dtype=torch.int32)
        self.offsets = offsets_of(torch.bincount(flat, minlength=E).numpy())
        self.token, self.inv = (order // K).to(torch.int32).cuda(), inv.cuda()
        self.idx = idx
        self.w = (torch.rand(T * K, generator=g) + 0.2).cuda()
        self.x, self.dout = randn(g, T, H), randn(g, T, H)
        self.gate, self.up, self.down = (randn(g, E, *s, scale=s[1] ** -0.5) for s in ((I, H), (I, H), (H, I)))
        P = T * K
        bf, f32 = dict(dtype=BF, device="cuda"), dict(dtype=F32, device="cuda")
        self.g, self.u, self.h, self.dh, self.dg, self.du = (torch.empty(P, I, **bf) for _ in range(6))
        self.y, self.dx_sorted = torch.empty(P, H, **f32), torch.empty(P, H, **f32)
        self.d_gate, self.d_up = torch.zeros(E, I, H, **f32), torch.zeros(E, I, H, **f32)
        self.d_down, self.dw = torch.zeros(E, H, I, **f32), torch.empty(P, **f32)
        self.out, self.dx = torch.empty(T, H, **bf), torch.empty(T, H, **bf)
        params = [self.gate, self.up, self.down]
        z = lambda: [torch.zeros(p.numel(), dtype=torch.uint8, device="cuda") for p in params]  # noqa: E731
        sc = lambda: [torch.zeros(-(-p.numel() // 128), **f32) for p in params]  # noqa: E731
        self.m, self.v, self.ms, self.vs = z(), z(), sc(), sc()
        self.master = [p.float() for p in params]
        self.step = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.plan = moe.MoEAdamWPlan(params, [self.d_gate, self.d_up, self.d_down], self.m, self.v, master=self.master,
                                     exp_avg_scale=self.ms, exp_avg_sq_scale=self.vs, weight_decay=0.01)

    def combine(self, rows, out):
        # moe_combine takes layer sizes (multiples of 128 and 64); this layer's are odd, so torch sums
        out.copy_(rows[self.inv.long()].view(self.T, self.K, -1).sum(1))

    def forward(self):
        moe.moe_grouped_gemm(self.x, self.gate, self.offsets, self.g, row_map=self.token)
        moe.moe_grouped_gemm(self.x, self.up, self.offsets, self.u, row_map=self.token)
        moe.moe_swiglu(self.g, self.u, self.h, limit=self.limit, row_w=self.w, pos=self.inv)
        moe.moe_grouped_gemm(self.h, self.down, self.offsets, self.y)

    def backward(self):
        moe.moe_grouped_gemm_dgrad(self.dout, self.down, self.offsets, self.dh, row_map=self.token)
        moe.moe_grouped_gemm_wgrad(self.dout, self.h, self.offsets, self.d_down, dy_map=self.token, accumulate=True)
        moe.moe_swiglu_backward(self.g, self.u, self.dh, self.dg, self.du, limit=self.limit, row_w=self.w, pos=self.inv, drow_w=self.dw)
        moe.moe_grouped_gemm_dgrad(self.dg, self.gate, self.offsets, self.dx_sorted, dy2=self.du, w2=self.up)
        moe.moe_grouped_gemm_wgrad(self.dg, self.x, self.offsets, self.d_gate, x_map=self.token, accumulate=True)
        moe.moe_grouped_gemm_wgrad(self.du, self.x, self.offsets, self.d_up, x_map=self.token, accumulate=True)

    def update(self):
        self.step.add_(1)
        moe.moe_adamw_step(self.plan, lr=1e-3, step=self.step, seed=9)

    def run(self):
        for t in (self.d_gate, self.d_up, self.d_down):
            t.zero_()
        self.forward()
        self.combine(self.y, self.out)
        self.backward()
        self.combine(self.dx_sorted, self.dx)
        self.update()

    def results(self):
        return [self.out, self.dx, self.dw, self.d_gate, self.d_up, self.d_down, self.gate, self.up, self.down, *self.m, *self.v,
                *self.ms, *self.vs, *self.master]


def layer64(s, x, gate, up, down, w):
    """The routed experts in float64, token by token and slot by slot."""
    out = torch.zeros(s.T, x.shape[1], dtype=torch.float64)
    for t in range(s.T):
        for k in range(s.K):
            e = int(s.idx[t, k])
            a = torch.nn.functional.silu(gate[e] @ x[t]) * (up[e] @ x[t])
            out[t] = out[t] + w[t * s.K + k] * (down[e] @ a.clamp(-s.limit, s.limit))
    return out


def test_training_step_of_a_layer():
    """All operators in turn against float64 autograd and a difference along a random direction.  On
    the way to any result at most six roundings to bf16 follow each other, each at most 2^-8 of its
    value; the 2-norm of a result may be off by twice their sum."""
    s = Step(30)
    leaves = [t.double().cpu().requires_grad_() for t in (s.x, s.gate, s.up, s.down, s.w)]
    loss_of = lambda *a: (layer64(s, *a) * s.dout.double().cpu()).sum()  # noqa: E731
    want = layer64(s, *leaves)
    (want * s.dout.double().cpu()).sum().backward()
    s.run()
    got = [s.dx, s.d_gate, s.d_up, s.d_down, s.dw]
    bound = 2 * 6 * HALF_BF16
    assert np.linalg.norm(f64(s.out) - want.detach().numpy()) <= bound * np.linalg.norm(want.detach().numpy())
    g = gen(31)
    for t, l in zip(got, leaves):
        assert np.linalg.norm(f64(t) - l.grad.numpy()) <= bound * np.linalg.norm(l.grad.numpy())
        d = torch.randn(l.shape, generator=g, dtype=torch.float64)
        e = 1e-6
        with torch.no_grad():
            moved = [[(o + sgn * e * d if o is l else o) for o in leaves] for sgn in (1, -1)]
            slope = ((loss_of(*moved[0]) - loss_of(*moved[1])) / (2 * e)).item()
        dot = float((f64(t) * d.numpy()).sum())
        # the direction's product errs by at most the gradient's error times the direction's length; the
        # values that the clamp's border crosses within e move the quotient by less than 1e-3 of it
        assert abs(dot - slope) <= bound * np.linalg.norm(l.grad.numpy()) * np.linalg.norm(d.numpy()) + 1e-3 * abs(slope)


def test_training_step_is_deterministic():
    a, b = Step(32), Step(32)
    a.run()
    b.run()
    for x, y in zip(a.results(), b.results()):
        assert torch.equal(x, y)


def test_training_steps_in_a_graph():
    """A captured step (its AdamW reading the step count from the device) replayed several times,
    with eager work between the replays, against the same steps run eagerly."""
    a, b = Step(33), Step(33)
    eager = Step(34)
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
        for x, y in zip(a.results(), b.results()):
            assert torch.equal(x, y)


def test_two_steps_on_two_streams():
    """Two layers' steps enqueued at once on two streams: the results of each alone."""
    solo = [Step(s, T=300) for s in (35, 36)]
    for s in solo:
        s.run()
    torch.cuda.synchronize()
    both = [Step(s, T=300) for s in (35, 36)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for s, st in zip(both, streams):
        with torch.cuda.stream(st):
            s.run()
    torch.cuda.synchronize()
    for s, t in zip(solo, both):
        for x, y in zip(s.results(), t.results()):
            assert torch.equal(x, y)


def test_given_stream_is_used():
    """stream= orders a call after that stream's work, not after the current one's."""
    st = torch.cuda.Stream()
    s = Step(37)
    torch.cuda.synchronize()
    big = torch.randn(4096, 4096, device="cuda")
    src = torch.zeros_like(s.x)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(5):
            big = big @ big
        src.copy_(s.x)                     # ready only after the products on `st`
    y = torch.empty_like(s.g)
    moe.moe_grouped_gemm(src, s.gate, s.offsets, y, row_map=s.token, stream=st)
    st.synchronize()
    s.forward()
    torch.cuda.synchronize()
    assert torch.equal(y, s.g)


def test_layer_with_shared_expert_matches_moe_forward():
    """The forward of the training operators, shared expert included, on the layer's own routing,
    dispatch and combine, against moe_forward.  Both round on the way (here gate, up and h to bf16,
    there h and y to fp16), so the outputs differ by at most twice four roundings of 2^-8 in the
    2-norm; the combine is moe_combine with weights of one."""
    from moe_case import cfg_for
    from synthetic import CONFIGS
    sc = CONFIGS["tiny"]
    cfg, T, H, I, E, K = cfg_for(sc), 50, sc.H, sc.I, sc.E, sc.K
    g = gen(38)
    x, rw = randn(g, T, H), randn(g, E, H, dtype=F32, scale=H ** -0.5)
    gate, up, down = randn(g, E, I, H, scale=H ** -0.5), randn(g, E, I, H, scale=H ** -0.5), randn(g, E, H, I, scale=I ** -0.5)
    sg, su, sd = randn(g, I, H, scale=H ** -0.5), randn(g, I, H, scale=H ** -0.5), randn(g, H, I, scale=I ** -0.5)
    ws = torch.empty(moe.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    want = torch.empty(T, H, dtype=BF, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, w = torch.empty(T, K, **i32), torch.empty(T, K, device="cuda")
    moe.moe_forward(cfg, T, x, rw, None, moe.MoEExpertWeights(gate, up, down, shared_gate=sg, shared_up=su, shared_down=sd),
                    want, idx, w, None, ws)
    P = T * K + T
    counts, off = torch.empty(E + 1, **i32), torch.empty(E + 2, **i32)
    token, inv = torch.empty(P, **i32), torch.empty(T, K, **i32)
    moe.moe_dispatch(cfg, T, idx, counts, off, token, inv, ws)
    gb, ub, hb = (torch.empty(P, I, dtype=BF, device="cuda") for _ in range(3))
    y = torch.empty(P, H, device="cuda")
    for o, wg, wu, wd in ((off[:E + 1], gate, up, down), (off[E:], sg[None], su[None], sd[None])):
        moe.moe_grouped_gemm(x, wg, o, gb, row_map=token)
        moe.moe_grouped_gemm(x, wu, o, ub, row_map=token)
    moe.moe_swiglu(gb, ub, hb, row_w=w.view(-1), pos=inv.view(-1))
    moe.moe_swiglu(gb[T * K:], ub[T * K:], hb[T * K:])
    for o, wd in ((off[:E + 1], down), (off[E:], sd[None])):
        moe.moe_grouped_gemm(hb, wd, o, y)
    out = torch.empty_like(want)
    moe.moe_combine(cfg, T, y, inv, torch.ones_like(w), out)
    assert np.linalg.norm(f64(out) - f64(want)) <= 2 * 4 * HALF_BF16 * np.linalg.norm(f64(want))
    moe.moe_update_expert_bias(cfg, counts, torch.zeros(E, device="cuda"), 1e-3)
    torch.cuda.synchronize()


def test_operands_and_results_side_by_side():
    """Input and output columns of one buffer, as a training program packs them."""
    g = gen(40)
    counts, N, K, C = [20, 7, 0, 40], 40, 72, 40
    off, P, o = offsets_of(counts), 67, offsets_of(counts).cpu().numpy()
    buf, w = randn(g, P, K + N + 3 * C), randn(g, 4, N, K)
    before = buf.clone()
    x, y = buf[:, :K], buf[:, K:K + N]
    moe.moe_grouped_gemm(x, w, off, y)
    check(y, *orc.grouped_forward(f64(x), f64(w), o, np.zeros((P, N))), K, True)
    gate, up, h = (buf[:, K + N + i * C:K + N + (i + 1) * C] for i in range(3))
    moe.moe_swiglu(gate, up, h)
    assert np.allclose(f64(h), orc.swiglu(f64(gate), f64(up), 0)[3], rtol=2.1 * HALF_BF16 / 2, atol=1e-6)
    keep = [slice(0, K), slice(K + N, K + N + 2 * C)]
    assert all(torch.equal(buf[:, k], before[:, k]) for k in keep)


def test_steps_from_two_host_threads():
    """Two threads, each with a stream and a layer of its own: the results of each alone."""
    import threading
    solo = [Step(s, T=200) for s in (41, 42)]
    for s in solo:
        s.run()
    torch.cuda.synchronize()
    both, failed = [Step(s, T=200) for s in (41, 42)], []
    torch.cuda.synchronize()

    def work(s):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                s.run()
            st.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in both]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for s, t in zip(solo, both):
        for x, y in zip(s.results(), t.results()):
            assert torch.equal(x, y)


@pytest.mark.slow
@pytest.mark.parametrize("skew", [0.0, 1.2])
def test_grouped_full_layer_sampled(skew):
    """512 groups of 768 x 2560 weights, 65,536 positions; sampled rows and whole sampled groups."""
    E, N, K, P, T = 512, 768, 2560, 65536, 8192
    gg = torch.Generator(device="cuda")
    gg.manual_seed(43)
    rnd = lambda *s: torch.randn(*s, generator=gg, device="cuda", dtype=torch.float32).to(BF)  # noqa: E731
    share = torch.exp(torch.randn(E, generator=gg, device="cuda") * skew)
    group = torch.multinomial(share, P, replacement=True, generator=gg).sort().values
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(group, minlength=E).cumsum(0)
    token = torch.randint(0, T, (P,), generator=gg, device="cuda", dtype=torch.int32)
    x, dy, w = rnd(T, K), rnd(P, N), rnd(E, N, K)
    y, dx = torch.empty(P, N, dtype=BF, device="cuda"), torch.empty(P, K, device="cuda")
    dw = torch.empty(E, N, K, device="cuda")
    moe.moe_grouped_gemm(x, w, off, y, row_map=token)
    moe.moe_grouped_gemm_dgrad(dy, w, off, dx)
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw, x_map=token)
    for p in [0, 1, P - 1, *torch.randint(0, P, (40,), generator=gg, device="cuda").tolist()]:
        e = int(group[p])
        we, xp, dp = f64(w[e]), f64(x[token[p].long()]), f64(dy[p])
        check(y[p], we @ xp, np.abs(we) @ np.abs(xp), K, True)
        check(dx[p], dp @ we, np.abs(dp) @ np.abs(we), N, False)
    o = off.tolist()
    sizes = np.diff(o)
    for e in {0, E - 1, int(sizes.argmax()), int(sizes.argmin()), 200}:
        d, xr = f64(dy[o[e]:o[e + 1]]), f64(x[token[o[e]:o[e + 1]].long()])
        check(dw[e], d.T @ xr, np.abs(d).T @ np.abs(xr), max(1, int(sizes[e])), False)


# ---- plans with empty tensors --------------------------------------------------------------------

@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
def test_adamw_with_an_empty_tensor_first(eight):
    """Master weights and an empty tensor before the others: the step of the same tensors without
    it, bit for bit (fp32 states), and every parameter the rounding of its master copy."""
    sizes = [0, 129, 0, 1000]
    a = adamw_inputs(13, BF, BF, eight, True, sizes)
    b = adamw_inputs(13, BF, BF, eight, True, sizes)
    mk = lambda t, keep: moe.MoEAdamWPlan(  # noqa: E731
        *([x for x, n in zip(t[i], sizes) if n or keep] for i in (0, 1, 3, 4)), master=[x for x, n in zip(t[2], sizes) if n or keep],
        **({k: [x for x, n in zip(t[i], sizes) if n or keep] for k, i in (("exp_avg_scale", 5), ("exp_avg_sq_scale", 6))} if eight else {}))
    pa, pb = mk(a, True), mk(b, False)
    old = [t.clone() for t in a[2]]
    for p in (pa, pb):
        moe.moe_adamw_step(p, lr=1e-2, step=1, seed=4)
    for i, n in enumerate(sizes):
        assert torch.equal(a[0][i], a[2][i].to(BF))
        # the parameters do not depend on the states' rounding after the first step
        assert torch.equal(a[2][i], b[2][i]) and (n == 0 or not torch.equal(a[2][i], old[i]))
        if not eight:
            assert torch.equal(a[3][i], b[3][i]) and torch.equal(a[4][i], b[4][i])


# ---- gradients of empty groups -------------------------------------------------------------------

@pytest.mark.parametrize("counts", [[0, 3, 0, 0, 70, 0], [0, 0, 0], [0] * 200 + [5] + [0] * 100], ids=["some", "none", "one_of_many"])
@pytest.mark.parametrize("dims", [(8, 8), (136, 264), (520, 776)], ids=str)
def test_wgrad_leaves_gradients_of_empty_groups(counts, dims):
    """Adding, an empty group's gradient keeps its bits: negative zeros, NaN payloads and infinities."""
    g = gen(50)
    N, K = dims
    off, P = offsets_of(counts, 1), 1 + sum(counts) + 2
    dy, x = randn(g, P, N), randn(g, P, K)
    bits = torch.randint(-2**31, 2**31 - 1, (len(counts), N, K), generator=g, dtype=torch.int64).to(torch.int32)
    bits[:, 0] = -2**31                                        # -0.0
    bits[:, 1] = torch.tensor(0x7F800001, dtype=torch.int32)   # a signalling NaN with a payload
    full = [e for e, c in enumerate(counts) if c]
    empty = [e for e, c in enumerate(counts) if not c]
    dw = bits.cuda().view(F32)
    dw[full] = randn(g, len(full), N, K, dtype=F32)
    before = dw.clone()
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw, accumulate=True)
    assert torch.equal(dw.view(torch.int32)[empty], before.view(torch.int32)[empty])
    o = off.cpu().numpy()
    for e in full:
        d, r = f64(dy)[o[e]:o[e + 1]], f64(x)[o[e]:o[e + 1]]
        check(dw[e], d.T @ r + f64(before[e]), np.abs(d).T @ np.abs(r) + np.abs(f64(before[e])), counts[e] + 1, False)


def test_vectors_between_the_rows_of_a_result():
    """Routing weights, positions and their gradient in the columns that a strided result leaves out."""
    g = gen(51)
    R, C, LD = 3, 16, 48
    buf = torch.zeros(R, LD, dtype=BF, device="cuda")
    h, dgate, dup = buf[:, :C], torch.zeros(R, LD, dtype=BF, device="cuda"), torch.zeros(R, LD, dtype=BF, device="cuda")
    w, pos = buf.view(F32)[0, 8:8 + R], buf.view(torch.int32)[1, 8:8 + R]
    drow = dgate.view(F32)[1, 8:8 + R]
    w.copy_(torch.rand(R, generator=g) + 0.1)
    pos.copy_(torch.tensor([2, 0, 1], dtype=torch.int32))
    gate, up, dh = randn(g, R, C), randn(g, R, C), randn(g, R, C)
    apart = [torch.empty(R, C, dtype=BF, device="cuda") for _ in range(3)] + [torch.empty(R, device="cuda")]
    moe.moe_swiglu(gate, up, apart[0], row_w=w.clone(), pos=pos.clone())
    moe.moe_swiglu_backward(gate, up, dh, apart[1], apart[2], row_w=w.clone(), pos=pos.clone(), drow_w=apart[3])
    moe.moe_swiglu(gate, up, h, row_w=w, pos=pos)
    moe.moe_swiglu_backward(gate, up, dh, dgate[:, :C], dup[:, :C], row_w=w, pos=pos, drow_w=drow)
    for got, want in zip((h, dgate[:, :C], dup[:, :C], drow), apart):
        assert torch.equal(got, want)


# ---- small and zero eps --------------------------------------------------------------------------

@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-30, 1e-20, 1e-15, 2.0 ** -40, 2.0 ** -39, 1e-8])
@pytest.mark.parametrize("pdt,master", [(BF, True), (F32, False)], ids=["bf16_master", "fp32"])
def test_adamw_small_gradients_and_eps(eps, pdt, master):
    """Gradients down to where the second moment is subnormal: the update still divides by its root.
    Zero gradients leave the parameters but for the decay, unless eps is zero too (then 0 / 0)."""
    g = gen(60)
    n, lr, betas, wd = 4096, 1e-2, (0.9, 0.999), 0.1
    size = torch.logspace(-20.9, 0, n, dtype=torch.float64).float()
    grad = (size * torch.sign(torch.randn(n, generator=g))).cuda()
    grad[::64] = 0.0
    param = [randn(g, n, dtype=pdt)]
    ms = [param[0].float()] if master else None
    m, v = ([torch.zeros(n, device="cuda")] for _ in range(2))
    plan = moe.MoEAdamWPlan(param, [grad], m, v, master=ms, weight_decay=wd)
    for step in (1, 2, 40):
        before = f64((ms or param)[0])
        wm, wv = orc.adamw_moments(m[0].cpu().numpy(), v[0].cpu().numpy(), grad.cpu().numpy(), betas)
        moe.moe_adamw_step(plan, lr=lr, step=step, betas=betas, eps=eps)
        assert np.array_equal(m[0].cpu().numpy(), wm) and np.array_equal(v[0].cpu().numpy(), wv)
        got = f64((ms or param)[0])
        with np.errstate(invalid="ignore", divide="ignore"):
            want = orc.adamw_param(before, wm, wv, lr, step, betas, float(np.float32(eps)), wd)
        zero = (wm == 0) & (wv == 0)
        assert zero.any() and (wv[~zero] > 0).all()
        assert (wv[~zero] < 2.0 ** -126).any()
        ok = ~zero if eps == 0.0 else np.ones(n, bool)
        assert np.isfinite(want[ok]).all()
        # about ten fp32 operations on the update and three on the parameter, as in test_adamw
        tol = 16 * U32 * (np.abs(want - before) + lr) + 4 * U32 * np.abs(before)
        assert (np.abs(got - want) <= tol)[ok].all()
        assert ok.all() or np.isnan(got[~ok]).all()
        if not ok.all():  # the elements without a gradient go on from where they were
            for t in (ms or []) + param:
                t[torch.from_numpy(~ok).cuda()] = 1.0


@pytest.mark.parametrize("step", [0, -3, -2**40])
@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
def test_adamw_device_step_below_one_writes_nothing(step, eight):
    """A step count that is read on the device is checked there: before the first step nothing moves."""
    params, grads, ms, m, v, sc, sv = adamw_inputs(61, BF, BF, eight, True)
    plan = moe.MoEAdamWPlan(params, grads, m, v, master=ms, exp_avg_scale=sc, exp_avg_sq_scale=sv, weight_decay=0.1)
    arrays = [t for ts in (params, ms, m, v, sc or [], sv or []) for t in ts]
    before = [t.clone() for t in arrays]
    at = torch.tensor([step], device="cuda")
    moe.moe_adamw_step(plan, lr=1e-2, step=at)
    for t, b in zip(arrays, before):
        assert torch.equal(t, b)
    at.fill_(1)
    moe.moe_adamw_step(plan, lr=1e-2, step=at)
    assert all(torch.isfinite(t).all() for t in params + ms)
    assert all(not torch.equal(t, b) for t, b in zip(params, before) if t.numel() >= 128)


# ---- a plan dropped while its step is still to run -----------------------------------------------

def two_plans_arrays():
    return [[torch.ones(20000, device="cuda")] for _ in range(4)]


@pytest.mark.parametrize("how", ["given", "current", "handle"])
def test_plan_table_outlives_a_plan_that_is_dropped(how):
    """A step on a stream of its own reads the plan's table after the plan is gone: the table's memory
    is not handed out again before that (addresses are compared, nothing is overwritten)."""
    arrays, want = two_plans_arrays(), two_plans_arrays()
    moe.moe_adamw_step(moe.MoEAdamWPlan(*want), lr=1e-2, step=1)
    st = torch.cuda.Stream()
    plan = moe.MoEAdamWPlan(*arrays)
    at, size = plan.image.data_ptr(), plan.image.numel()
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(20):                # the step waits behind these
            big = big @ big
    if how == "current":
        with torch.cuda.stream(st):
            moe.moe_adamw_step(plan, lr=1e-2, step=1)
    else:
        moe.moe_adamw_step(plan, lr=1e-2, step=1, stream=st if how == "given" else st.cuda_stream)
    del plan
    busy = not st.query()
    taken = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    if busy:
        assert all(t.data_ptr() != at for t in taken)
    torch.cuda.synchronize()
    assert busy, "the products ended before the step was enqueued"
    for a, b in zip(arrays, want):
        assert torch.equal(a[0], b[0])


# ---- the range of the 8-bit states ---------------------------------------------------------------

@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e25], ids=str)
def test_adamw_nonfinite_block_is_not_finite_in_both_moments(bad):
    """Every value of a block with an infinite or NaN moment reads back as not finite (1e25: only its
    square is infinite), every value of the blocks beside it as finite, and stays so at the next step."""
    params, grads, _, m, v, sc, sv = adamw_inputs(12, BF, F32, True, False, [512])
    grads[0][130] = bad
    plan = moe.MoEAdamWPlan(params, grads, m, v, exp_avg_scale=sc, exp_avg_sq_scale=sv)
    for step in (1, 2):
        moe.moe_adamw_step(plan, lr=1e-3, step=step)
        for codes, scales, signed in ((m[0], sc[0], True), (v[0], sv[0], False)):
            out = torch.empty(512, device="cuda")
            moe.moe_adamw_dequantise(codes, scales, out, signed)
            hit = torch.isfinite(out[128:256])
            assert hit.all() if signed and bad == 1e25 else not hit.any()
            assert torch.isfinite(out[:128]).all() and torch.isfinite(out[256:]).all()
        grads[0][130] = 0.01
        fine = torch.cat([params[0][:128], params[0][256:]])
        assert torch.isfinite(fine).all()


@pytest.mark.parametrize("ratio", [0.25, 0.9, 1.03, 1.0625, 1.2, 3.0, 1000.0])
def test_adamw_state_range(ratio):
    """What a block keeps of values far below its largest, in one step with beta1 = beta2 = 0 (the
    moments are g and g^2): a first moment up to 2^-15 of the scale is zero, so its parameter stays
    where it is, rising to unbiased at 1.125 2^-15; a second moment below 2^-31 is raised to it.  The
    bound is that of the rounding's mean over N values (two outcomes `apart` from each other)."""
    blocks, N = 400, 400 * 127
    low = 2.0 ** -15
    g = torch.full((blocks, 128), ratio * low, device="cuda")
    g[:, 0] = 1.875
    p = [torch.ones(blocks * 128, device="cuda")]
    m, v = ([torch.zeros(blocks * 128, dtype=torch.uint8, device="cuda")] for _ in range(2))
    sc, sv = ([torch.zeros(blocks, device="cuda")] for _ in range(2))
    plan = moe.MoEAdamWPlan(p, [g.view(-1)], m, v, exp_avg_scale=sc, exp_avg_sq_scale=sv)
    moe.moe_adamw_step(plan, lr=0.0, step=1, betas=(0.0, 0.0), seed=8)
    out = torch.empty(blocks * 128, device="cuda")
    moe.moe_adamw_dequantise(m[0], sc[0], out, True)
    got = out.view(blocks, 128)[:, 1:].double()
    value = float(g[0, 1])
    want = 0.0 if ratio <= 1 else 9 * (ratio - 1) * low if ratio < 1.125 else value
    apart = 0.0 if ratio <= 1 else 1.125 * low if ratio < 1.125 else value / 8
    assert abs(got.mean().item() - want) <= 5 * apart / 2 / N ** 0.5 + apart * 2.0 ** -16 + 9 * 2.0 ** -22 * value
    moe.moe_adamw_dequantise(v[0], sv[0], out, False)
    got, scale = out.view(blocks, 128)[:, 1:].double(), 1.875
    value = float(g[0, 1]) ** 2
    want = max(value, scale * 2.0 ** -31)
    apart = value / 8 if want == value else 0.0
    assert abs(got.mean().item() - want) <= 5 * apart / 2 / N ** 0.5 + apart * 2.0 ** -16 + 9 * 2.0 ** -22 * want
    if ratio <= 1:                        # the next step's first moment is all that would move it
        g[:, 1:] = 0.0
        moe.moe_adamw_step(plan, lr=1e-2, step=2, betas=(0.5, 0.999), seed=8)
        assert (p[0].view(blocks, 128)[:, 1:] == 1).all()


# ---- the shared expert on its own rows -----------------------------------------------------------

@pytest.mark.parametrize("T", [1, 50, 300])
def test_shared_expert_on_its_own_rows(T):
    """Forward, gradients and weight gradients of the shared expert from row T*K of the dispatch's
    buffers on, some slots routed nowhere: the float64 definitions, and the same as the calls on the
    whole buffers with the dispatch's own offsets and map; the routed experts' rows are left alone."""
    from moe_case import cfg_for
    from synthetic import CONFIGS
    sc = CONFIGS["tiny"]
    cfg, H, I, E, K = cfg_for(sc), sc.H, sc.I, sc.E, sc.K
    g = gen(70)
    P, s = T * K + T, T * K
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).to(torch.int32)
    idx[::5, 0] = -1                       # pairs that the dispatch ignores
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, off = torch.empty(E + 1, **i32), torch.empty(E + 2, **i32)
    token, inv = torch.empty(P, **i32), torch.empty(T, K, **i32)
    ws = torch.empty(moe.moe_workspace_size(cfg, T), dtype=torch.uint8, device="cuda")
    moe.moe_dispatch(cfg, T, idx.cuda(), counts, off, token, inv, ws)
    assert off[E:].tolist() == [s, P] and token[s:].tolist() == list(range(T))
    x, dout = randn(g, T, H), randn(g, T, H)
    wg, wu, wd = randn(g, 1, I, H, scale=H ** -0.5), randn(g, 1, I, H, scale=H ** -0.5), randn(g, 1, H, I, scale=I ** -0.5)
    own, one = offsets_of([T]), np.array([0, T])

    def buffers():
        bf = [torch.full((P, I), 3.0, dtype=BF, device="cuda") for _ in range(6)]
        return bf + [torch.full((P, H), 3.0, device="cuda") for _ in range(2)] + [torch.ones_like(t, dtype=F32) for t in (wg, wu, wd)]

    a, b = buffers(), buffers()
    for whole, (gb, ub, hb, dhb, dgb, dub, y, dx, d_gate, d_up, d_down) in ((False, a), (True, b)):
        v, o, m = (lambda t: t, off[E:], token) if whole else (lambda t: t[s:], own, None)
        moe.moe_grouped_gemm(x, wg, o, v(gb), row_map=m)
        moe.moe_grouped_gemm(x, wu, o, v(ub), row_map=m)
        moe.moe_swiglu(gb[s:], ub[s:], hb[s:], limit=2.0)
        moe.moe_grouped_gemm(v(hb), wd, o, v(y))
        moe.moe_grouped_gemm_dgrad(dout, wd, o, v(dhb), row_map=m)
        moe.moe_grouped_gemm_wgrad(dout, v(hb), o, d_down, dy_map=m, accumulate=True)
        moe.moe_swiglu_backward(gb[s:], ub[s:], dhb[s:], dgb[s:], dub[s:], limit=2.0)
        moe.moe_grouped_gemm_dgrad(v(dgb), wg, o, v(dx), dy2=v(dub), w2=wu)
        moe.moe_grouped_gemm_wgrad(v(dgb), x, o, d_gate, x_map=m, accumulate=True)
        moe.moe_grouped_gemm_wgrad(v(dub), x, o, d_up, x_map=m, accumulate=True)
    for t in a[:8]:
        assert (t[:s] == 3.0).all()
    X, DO, WG, WU, WD = (f64(t) for t in (x, dout, wg, wu, wd))
    for gb, ub, hb, dhb, dgb, dub, y, dx, d_gate, d_up, d_down in (a, b):
        z = np.zeros
        check(gb[s:], *orc.grouped_forward(X, WG, one, z((T, I))), H, True)
        check(ub[s:], *orc.grouped_forward(X, WU, one, z((T, I))), H, True)
        check(y[s:], *orc.grouped_forward(f64(hb)[s:], WD, one, z((T, H))), I, False)
        check(dhb[s:], *orc.grouped_dgrad(DO, WD, one, z((T, I))), H, True)
        check(dx[s:], *orc.grouped_dgrad(f64(dgb)[s:], WG, one, z((T, H)), None, f64(dub)[s:], WU), 2 * I, False)
        for dw, d, r in ((d_gate, f64(dgb)[s:], X), (d_up, f64(dub)[s:], X), (d_down, DO, f64(hb)[s:])):
            check(dw, *orc.grouped_wgrad(d, r, one, np.ones(dw.shape), None, None, True), T + 1, False)


# ---- offsets outside the positions ---------------------------------------------------------------

@pytest.mark.parametrize("raw", [[-5, 3, 20, 20, 400], [0, 0, 60, 2**31 - 1, 2**31 - 1], [-2**31, -1, 0, 61, 62], [70, 80, 90, 100, 110]], ids=str)
@pytest.mark.parametrize("mapped", [False, True])
def test_grouped_offsets_are_clamped(raw, mapped):
    """Offsets are taken as clamped to [0, rows]: groups end with the positions, rows of no group stay."""
    g = gen(80)
    P, N, K, G = 61, 40, 72, 4
    off = torch.tensor(raw, dtype=torch.int32).cuda()
    o = np.clip(np.array(raw, dtype=np.int64), 0, P)
    T = 9 if mapped else P
    m = torch.randint(-1, T + 1, (P,), generator=g, dtype=torch.int32).cuda() if mapped else None
    mn = None if m is None else m.cpu().numpy()
    x, dy, w = randn(g, T, K), randn(g, T, N), randn(g, G, N, K)
    y, dx, dw = randn(g, P, N, dtype=F32), randn(g, P, K, dtype=F32), randn(g, G, N, K, dtype=F32)
    by, bx, bw = f64(y), f64(dx), f64(dw)
    moe.moe_grouped_gemm(x, w, off, y, row_map=m)
    moe.moe_grouped_gemm_dgrad(dy, w, off, dx, row_map=m)
    moe.moe_grouped_gemm_wgrad(dy, x, off, dw, dy_map=m, x_map=m, accumulate=True)
    check(y, *orc.grouped_forward(f64(x), f64(w), o, by, mn), K, False)
    check(dx, *orc.grouped_dgrad(f64(dy), f64(w), o, bx, mn), N, False)
    check(dw, *orc.grouped_wgrad(f64(dy), f64(x), o, bw, mn, mn, True), P + 1, False)


# ---- elements past 32 bits -----------------------------------------------------------------------

def test_swiglu_rows_past_four_gibibytes():
    """Rows far apart in buffers of more than 4 GiB, forward and backward."""
    g = gen(90)
    R, LD, C = 700, 1 << 22, 40
    buf, out = (torch.empty(R, LD, dtype=BF, device="cuda") for _ in range(2))     # 5.9 GB each
    gate, up, dh = buf[:, 8:8 + C], buf[:, 128:128 + C], buf[:, 1 << 20:(1 << 20) + C]
    for t in (gate, up, dh):
        t.copy_(randn(g, R, C))
    pos, w = torch.randperm(R, generator=g).to(torch.int32).cuda(), (torch.rand(R, generator=g) + 0.1).cuda()
    h, dgate, dup = out[:, :C], out[:, 64:64 + C], out[:, 128:128 + C]
    drow, drow2 = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    moe.moe_swiglu(gate, up, h, limit=2.0, row_w=w, pos=pos)
    moe.moe_swiglu_backward(gate, up, dh, dgate, dup, limit=2.0, row_w=w, pos=pos, drow_w=drow)
    near = [t.contiguous() for t in (gate, up, dh)] + [torch.empty(R, C, dtype=BF, device="cuda") for _ in range(3)]
    moe.moe_swiglu(near[0], near[1], near[3], limit=2.0, row_w=w, pos=pos)
    moe.moe_swiglu_backward(near[0], near[1], near[2], near[4], near[5], limit=2.0, row_w=w, pos=pos, drow_w=drow2)
    for a, b in ((h, near[3]), (dgate, near[4]), (dup, near[5]), (drow, drow2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("eight", [False, True], ids=["s32", "s8"])
def test_adamw_tensor_past_two_to_the_32_values(eight):
    """One tensor of more than 2^32 values: its first and last values take the step of a small tensor
    (8 bits: one that holds the same blocks; read-outs within a code, at most 1/8, of the moments)."""
    n, tail, lr = (1 << 32) + 8192 + 77, 8192 + 77, 1e-2
    g = gen(91)
    small = randn(g, 2 * 8192 + 77, dtype=BF, scale=0.05), randn(g, 2 * 8192 + 77, dtype=BF, scale=1e-2)
    p, gr = (torch.zeros(n, dtype=BF, device="cuda") for _ in range(2))                # 8.6 GB each
    for big, s in zip((p, gr), small):
        big[:8192], big[-tail:] = s[:8192], s[8192:]
    z = lambda k: torch.zeros(k, dtype=torch.uint8 if eight else F32, device="cuda")  # noqa: E731
    m, v, ms, vs = z(n), z(n), z(len(small[0])), z(len(small[0]))
    sc = lambda k: [torch.zeros(-(-k // 128), device="cuda") for _ in range(2)] if eight else [None, None]  # noqa: E731
    big_sc, small_sc = sc(n), sc(len(small[0]))
    kw = lambda s: dict(exp_avg_scale=[s[0]], exp_avg_sq_scale=[s[1]]) if eight else {}  # noqa: E731
    moe.moe_adamw_step(moe.MoEAdamWPlan([p], [gr], [m], [v], **kw(big_sc)), lr=lr, step=1, seed=3)
    want = small[0].clone()
    moe.moe_adamw_step(moe.MoEAdamWPlan([want], [small[1]], [ms], [vs], **kw(small_sc)), lr=lr, step=1, seed=3)
    assert torch.equal(p[:8192], want[:8192]) and torch.equal(p[-tail:], want[8192:])
    assert not p[8192:16384].any() and not p[-tail - 8192:-tail].any()
    if not eight:
        for a, b in ((m, ms), (v, vs)):
            assert torch.equal(a[:8192], b[:8192]) and torch.equal(a[-tail:], b[8192:])
        return
    assert torch.equal(m[:8192], ms[:8192]) and torch.equal(v[:8192], vs[:8192])
    wm, wv = orc.adamw_moments(np.zeros(tail), np.zeros(tail), small[1][8192:].float().cpu().numpy(), (0.9, 0.999))
    for codes, scales, signed, x in ((m, big_sc[0], True, wm), (v, big_sc[1], False, wv)):
        assert torch.equal(scales[-65:], (small_sc[0] if signed else small_sc[1])[-65:])
        out = torch.empty(n, device="cuda")                                            # 17 GB
        moe.moe_adamw_dequantise(codes, scales, out, signed)
        got, floor = f64(out[-tail:]), np.repeat(scales[-65:].cpu().numpy(), 128)[:tail] * 1.125 * 2.0 ** -15
        assert (np.abs(got - x) <= np.abs(x) / 8 * (1 + 2.0 ** -20) + floor).all()
        assert not out[8192:16384].any()
        del out
