"""The training operators without a GPU: their definitions, and what the host layer refuses before
anything is enqueued (addresses given here are never dereferenced)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import sparse_moe_layer_bailingmoev3_amd as moe
from oracle import train_oracle as orc

needs_lib = pytest.mark.skipif(not os.path.exists(moe.lib_path()), reason="libmoe.so not built")

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = -1, -2, -3, -4
A = 1 << 40                                # an aligned address


def at(i):
    return A + (i << 36)                   # far enough apart for every size below


def groups(**kw):
    d = dict(groups=4, out_features=64, in_features=128, rows=100, offsets=at(0))
    d.update(kw)
    return moe._Groups(**d)


def rows(i, cols, **kw):
    d = dict(data=at(i), rows=100, ld=cols, row_map=None)
    d.update(kw)
    return moe._Rows(**d)


def forward(g=None, x=None, w=at(2), y=at(3), ldy=64, dtype=0, acc=0):
    g, x = g or groups(), x or rows(1, 128)
    return moe.load_library().moe_grouped_gemm(ctypes.byref(g), ctypes.byref(x), w, y, ldy, dtype, acc, None)


def dgrad(g=None, dy=None, w=at(2), dy2=None, w2=None, dx=at(3), ld=128, dtype=0, acc=0):
    g, dy = g or groups(), dy or rows(1, 64)
    return moe.load_library().moe_grouped_gemm_dgrad(ctypes.byref(g), ctypes.byref(dy), w, ctypes.byref(dy2) if dy2 else None, w2,
                                                     dx, ld, dtype, acc, None)


def wgrad(g=None, dy=None, x=None, dw=at(3), dtype=0, acc=0):
    g, dy, x = g or groups(), dy or rows(1, 64), x or rows(2, 128)
    return moe.load_library().moe_grouped_gemm_wgrad(ctypes.byref(g), ctypes.byref(dy), ctypes.byref(x), dw, dtype, acc, None)


@needs_lib
@pytest.mark.parametrize("call,code,words", [
    (lambda: forward(groups(groups=0)), INVALID, b"groups 0"),
    (lambda: forward(groups(groups=1026)), UNSUPPORTED, b"above 1025"),
    (lambda: forward(groups(out_features=60)), UNSUPPORTED, b"multiples of 8"),
    (lambda: forward(groups(in_features=0)), INVALID, b">= 1"),
    (lambda: forward(groups(in_features=65544)), UNSUPPORTED, b"above 65536"),
    (lambda: forward(groups(rows=-1)), INVALID, b">= 0"),
    (lambda: forward(groups(rows=2**31 - 1)), UNSUPPORTED, b"32-bit"),
    (lambda: forward(groups(offsets=None)), INVALID, b"offsets must not be NULL"),
    (lambda: forward(groups(offsets=at(0) + 2)), ALIGNMENT, b"offsets"),
    (lambda: forward(x=rows(1, 128, rows=99)), INVALID, b"without a row map"),
    (lambda: forward(x=rows(1, 128, ld=120)), INVALID, b"row stride"),
    (lambda: forward(x=rows(1, 128, ld=132)), UNSUPPORTED, b"multiple of 8"),
    (lambda: forward(x=rows(1, 128, data=None)), INVALID, b"x must not be NULL"),
    (lambda: forward(x=rows(1, 128, data=at(1) + 8)), ALIGNMENT, b"x is not"),
    (lambda: forward(x=rows(1, 128, row_map=at(4) + 1)), ALIGNMENT, b"row_map"),
    (lambda: forward(w=None), INVALID, b"w must not be NULL"),
    (lambda: forward(y=at(3) + 4), ALIGNMENT, b"y is not"),
    (lambda: forward(ldy=56), INVALID, b"row stride"),
    (lambda: forward(dtype=2), INVALID, b"dtype 2"),
    (lambda: forward(acc=1), UNSUPPORTED, b"accumulation needs fp32"),
    (lambda: forward(y=at(1)), INVALID, b"y overlaps x"),
    (lambda: forward(y=at(2) + 4 * 64 * 128 * 2 - 16), INVALID, b"y overlaps w"),
    (lambda: dgrad(dy2=rows(5, 64)), INVALID, b"together"),
    (lambda: dgrad(w2=at(6)), INVALID, b"together"),
    (lambda: dgrad(dy2=rows(5, 64, ld=8), w2=at(6)), INVALID, b"dy2"),
    (lambda: dgrad(dy2=rows(5, 64, ld=72), w2=at(6)), INVALID, b"same rows, row stride and row map"),
    (lambda: forward(groups(out_features=65536, in_features=32768)), UNSUPPORTED, b"4 GiB"),
    (lambda: forward(x=rows(1, 128, ld=(1 << 22) + 8)), UNSUPPORTED, b"row stride"),
    (lambda: dgrad(dy2=rows(5, 64), w2=at(6), dx=at(6)), INVALID, b"dx overlaps w2"),
    (lambda: forward(x=rows(1, 128, ld=256), y=at(1) + 240, ldy=256), INVALID, b"y overlaps x"),
    (lambda: forward(x=rows(1, 128, ld=256), y=at(1) + 400, ldy=256), INVALID, b"y overlaps x"),
    (lambda: wgrad(x=rows(2, 128, rows=50)), INVALID, b"x: 50 rows"),
    (lambda: wgrad(dw=at(2)), INVALID, b"dw overlaps x"),
    (lambda: wgrad(acc=1), UNSUPPORTED, b"accumulation needs fp32"),
    (lambda: wgrad(dw=None), INVALID, b"dw must not be NULL"),
])
def test_grouped_refusals(call, code, words):
    assert call() == code
    assert words in moe.load_library().moe_last_error()


@needs_lib
def test_no_positions_is_a_no_op():
    assert forward(groups(rows=0)) == 0 and dgrad(groups(rows=0)) == 0
    assert moe.load_library().moe_last_error() == b""


def swiglu(n=10, R=10, C=64, limit=0.0, gate=at(1), up=at(2), ld=64, w=None, pos=None, h=at(3), ldh=64):
    return moe.load_library().moe_swiglu(n, R, C, limit, gate, up, ld, w, pos, h, ldh, None)


def swiglu_bwd(n=10, R=10, C=64, dh=at(3), lddh=64, dgate=at(4), dup=at(5), ldd=64, dw=None):
    return moe.load_library().moe_swiglu_backward(n, R, C, 0.0, at(1), at(2), 64, dh, lddh, None, None, dgate, dup, ldd, dw, None)


@needs_lib
@pytest.mark.parametrize("call,code,words", [
    (lambda: swiglu(n=-1), INVALID, b">= 0"),
    (lambda: swiglu(n=2**31), UNSUPPORTED, b"32-bit"),
    (lambda: swiglu(C=0), INVALID, b"cols 0"),
    (lambda: swiglu(C=60, ld=64), UNSUPPORTED, b"multiple of 8"),
    (lambda: swiglu(limit=float("nan")), INVALID, b"NaN"),
    (lambda: swiglu(n=11), INVALID, b"without positions"),
    (lambda: swiglu(ld=56), INVALID, b"row stride"),
    (lambda: swiglu(gate=None), INVALID, b"gate"),
    (lambda: swiglu(up=at(2) + 2), ALIGNMENT, b"up"),
    (lambda: swiglu(h=at(1)), INVALID, b"h overlaps gate"),
    (lambda: swiglu(w=at(6) + 2), ALIGNMENT, b"row_w"),
    (lambda: swiglu_bwd(dh=None), INVALID, b"dh"),
    (lambda: swiglu_bwd(dgate=at(3)), INVALID, b"dgate overlaps dh"),
    (lambda: swiglu_bwd(dup=at(4)), INVALID, b"dgate overlaps dup"),
    (lambda: swiglu_bwd(dup=at(4) + 112, ldd=128), INVALID, b"dgate overlaps dup"),
    (lambda: swiglu_bwd(dw=at(6) + 1), ALIGNMENT, b"drow_w"),
])
def test_swiglu_refusals(call, code, words):
    assert call() == code
    assert words in moe.load_library().moe_last_error()


def adamw_tensor(i, n=1000, **kw):
    d = dict(param=at(10 * i + 1), grad=at(10 * i + 2), exp_avg=at(10 * i + 3), exp_avg_sq=at(10 * i + 4), numel=n)
    d.update(kw)
    return moe._AdamWTensor(**d)


def plan(tensors, pd=0, gd=0, st=0, image=True, short=0):
    lib, p = moe.load_library(), moe._AdamWPlan()
    arr = (moe._AdamWTensor * max(1, len(tensors)))(*tensors)
    rc = lib.moe_adamw_plan(len(tensors), ctypes.byref(arr), pd, gd, st, ctypes.byref(p), None, 0)
    if rc or not image:
        return rc, p, None
    buf = ctypes.create_string_buffer(p.image_bytes)
    return lib.moe_adamw_plan(len(tensors), ctypes.byref(arr), pd, gd, st, ctypes.byref(p), buf, p.image_bytes - short), p, buf


@needs_lib
@pytest.mark.parametrize("call,code,words", [
    (lambda: plan([adamw_tensor(0, n=-1)]), INVALID, b"numel"),
    (lambda: plan([adamw_tensor(0, n=1 << 41)]), UNSUPPORTED, b"too large"),
    (lambda: plan([adamw_tensor(0, param=None)]), INVALID, b"tensor 0: param"),
    (lambda: plan([adamw_tensor(0), adamw_tensor(1, grad=at(12) + 8)]), ALIGNMENT, b"tensor 1: grad"),
    (lambda: plan([adamw_tensor(0, weight_decay=float("nan"))]), INVALID, b"weight_decay"),
    (lambda: plan([adamw_tensor(0)], pd=2), INVALID, b"dtype 2"),
    (lambda: plan([adamw_tensor(0)], st=2), INVALID, b"state_format"),
    (lambda: plan([adamw_tensor(0, master=at(5))], pd=1), INVALID, b"master"),
    (lambda: plan([adamw_tensor(0, master=at(5)), adamw_tensor(1)]), INVALID, b"for all tensors or for none"),
    (lambda: plan([adamw_tensor(0)], st=1), INVALID, b"exp_avg_scale"),
    (lambda: plan([adamw_tensor(0), adamw_tensor(1, param=at(1) + 1984)]), INVALID, b"overlaps"),
    (lambda: plan([adamw_tensor(0), adamw_tensor(0)]), INVALID, b"overlaps"),
    (lambda: plan([adamw_tensor(0, exp_avg_sq=at(3))]), INVALID, b"overlaps"),
    (lambda: plan([adamw_tensor(0)], short=1), WORKSPACE, b"plan image"),
])
def test_adamw_plan_refusals(call, code, words):
    assert call()[0] == code
    assert words in moe.load_library().moe_last_error()


@needs_lib
def test_adamw_plan_shares_gradients_and_counts_chunks():
    rc, p, _ = plan([adamw_tensor(0, n=8193), adamw_tensor(1, n=0), adamw_tensor(2, n=1, grad=at(2))])
    assert rc == 0 and p.n_tensors == 3 and p.n_chunks == 3


@needs_lib
@pytest.mark.parametrize("kw,words", [
    (dict(beta1=1.0), b"beta1"), (dict(beta2=-0.1), b"beta2"), (dict(eps=-1.0), b"eps"), (dict(lr=float("inf")), b"lr"),
    (dict(step=0), b"step"),
])
def test_adamw_step_refusals(kw, words):
    _, p, _ = plan([adamw_tensor(0)])
    d = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1)
    d.update(kw)
    cfg = moe._AdamWConfig(**d)
    assert moe.load_library().moe_adamw_step(ctypes.byref(cfg), ctypes.byref(p), at(9), None) == INVALID
    assert words in moe.load_library().moe_last_error()


# ---- the binding's own checks --------------------------------------------------------------------

def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


def u8(n):
    return torch.zeros(n, dtype=torch.uint8)


OFF = i32(0, 2, 4)


@needs_lib
@pytest.mark.parametrize("call,words", [
    (lambda: moe.moe_grouped_gemm(bf(4, 16), bf(2, 8, 16), OFF, bf(4, 8)), "must lie on a GPU"),
    (lambda: moe.moe_grouped_gemm(bf(4, 16), bf(2, 8, 24), OFF, bf(4, 8)), "x has 16 columns, 24 needed"),
    (lambda: moe.moe_grouped_gemm(bf(4, 16), bf(2, 8, 16), i32(0, 4), bf(4, 8)), "offsets has 2 entries, 3 needed"),
    (lambda: moe.moe_grouped_gemm(bf(4, 16), bf(2, 8, 16), OFF.long(), bf(4, 8)), "offsets must be torch.int32"),
    (lambda: moe.moe_grouped_gemm(bf(4, 16).float(), bf(2, 8, 16), OFF, bf(4, 8)), "x must be torch.bfloat16"),
    (lambda: moe.moe_grouped_gemm(bf(4, 16), bf(2, 16, 8).transpose(1, 2), OFF, bf(4, 8)), "w must be contiguous"),
    (lambda: moe.moe_grouped_gemm(bf(16, 4).t(), bf(2, 8, 16), OFF, bf(4, 8)), "side by side"),
    (lambda: moe.moe_grouped_gemm(bf(4, 16), bf(2, 8, 16), OFF, bf(4, 8), row_map=i32(0, 1)), "row map of x has 2 entries"),
    (lambda: moe.moe_grouped_gemm(bf(4, 16), bf(2, 8, 16), OFF, bf(4, 16)), "y has 16 columns, w makes 8"),
    (lambda: moe.moe_grouped_gemm(bf(4, 16), bf(2, 8, 16), OFF, bf(4, 8).half()), "y must be bfloat16 or float32"),
    (lambda: moe.moe_grouped_gemm(bf(4, 16), bf(8, 16), OFF, bf(4, 8)), "w must have 3 dimension"),
    (lambda: moe.moe_grouped_gemm(bf(4, 16), None, OFF, bf(4, 8)), "w must be a tensor"),
    (lambda: moe.moe_grouped_gemm(bf(4, 16), bf(2, 8, 16), OFF, bf(4, 8), stream=torch.device("cpu")), "must lie on a GPU"),
    (lambda: moe.moe_grouped_gemm_dgrad(bf(4, 8), bf(2, 8, 16), OFF, bf(4, 16), dy2=bf(4, 8)), "given together"),
    (lambda: moe.moe_grouped_gemm_dgrad(bf(4, 8), bf(2, 8, 16), OFF, bf(4, 16), dy2=bf(4, 8), w2=bf(2, 16, 16)), "w2 is"),
    (lambda: moe.moe_grouped_gemm_dgrad(bf(4, 8), bf(2, 8, 16), OFF, bf(4, 8)), "dx has 8 columns"),
    (lambda: moe.moe_grouped_gemm_wgrad(bf(4, 8), bf(5, 16), OFF, bf(2, 8, 16)), "different numbers of positions"),
    (lambda: moe.moe_grouped_gemm_wgrad(bf(4, 8), bf(4, 24), OFF, bf(2, 8, 16)), "x has 24 columns"),
    (lambda: moe.moe_swiglu(bf(4, 8), bf(4, 16), bf(4, 8)), "up is [4, 16], gate is [4, 8]"),
    (lambda: moe.moe_swiglu(bf(4, 8), bf(4, 16)[:, :8], bf(4, 8)), "same row stride"),
    (lambda: moe.moe_swiglu(bf(4, 8), bf(4, 8), bf(4, 8), row_w=torch.zeros(3), pos=i32(0, 1)), "row_w has 3 entries, 2 needed"),
    (lambda: moe.moe_swiglu_backward(bf(4, 8), bf(4, 8), bf(4, 8), bf(4, 8), bf(4, 16)[:, :8]), "dgate and dup"),
    (lambda: moe.moe_swiglu_backward(bf(4, 8), bf(4, 8), bf(4, 8), bf(4, 8), bf(4, 8), drow_w=torch.zeros(3)), "drow_w has 3"),
    (lambda: moe.MoEAdamWPlan([bf(8)], [bf(9)], [bf(8).float()], [bf(8).float()]), "grads[0] has 9 values, 8 needed"),
    (lambda: moe.MoEAdamWPlan([bf(8)], [bf(8)], [bf(8).float()], [bf(8)]), "exp_avg_sq[0] must be torch.float32"),
    (lambda: moe.MoEAdamWPlan([bf(8)], [bf(8)], [u8(8)], [u8(8)]), "scales belong to uint8 states"),
    (lambda: moe.MoEAdamWPlan([bf(8)], [bf(8)], [bf(8).float()], [bf(8).float()]), "one GPU must hold them all"),
    (lambda: moe.MoEAdamWPlan([], [], [], []), "params must not be empty"),
    (lambda: moe.moe_adamw_dequantise(u8(129), torch.zeros(1), torch.zeros(129), True), "scales has 1 entries, 2 needed"),
])
def test_binding_refusals(call, words):
    with pytest.raises(moe.MoEError) as e:
        call()
    assert e.value.status in (INVALID, UNSUPPORTED)
    assert words in str(e.value)


# ---- the definitions -----------------------------------------------------------------------------

@pytest.mark.parametrize("signed", [True, False])
def test_state_code_decodes_to_a_neighbour(signed):
    """A code stands for one of the two representable values next to what it encodes."""
    r = np.random.RandomState(0)
    x = (r.randn(1000) * np.exp(r.randn(1000) * 2)).astype(np.float32)
    x = x if signed else x * x
    c, s = orc.state_encode(x, signed, 3, 1, 2)
    d = orc.state_decode(c, s, signed).astype(np.float64)
    big = np.abs(x) >= np.repeat(s, 128)[:1000] * 2.0 ** -14
    # neighbours are 1/8 to 1/16 of the value apart
    assert (np.abs(d - x) <= np.abs(x) / 8 * (1 + 1e-6))[big].all()
    assert (d[~big] >= 0).all() or signed
    top = np.abs(x[:896]).reshape(7, 128).argmax(1) + 128 * np.arange(7)
    assert np.allclose(d[top], x[top], rtol=2.0 ** -22)


def test_state_rounding_is_unbiased_over_seeds():
    x = np.full(128, 0.3, np.float32)
    x[0] = 1.0
    got = np.mean([orc.state_decode(*orc.state_encode(x, True, 0, s, 1), True)[1:].mean() for s in range(200)])
    # 200 x 127 roundings, each off by at most 0.3 / 8: five standard deviations are 0.0012
    assert abs(got - 0.3) < 0.0012


def test_adamw_definition_matches_torch():
    """The definition against torch's own AdamW, three steps in float64 parameters."""
    r = np.random.RandomState(1)
    p0, gs = r.randn(50), [r.randn(50).astype(np.float32) for _ in range(3)]
    t = torch.nn.Parameter(torch.tensor(p0))
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
    p, m, v = p0.copy(), np.zeros(50, np.float32), np.zeros(50, np.float32)
    for i, g in enumerate(gs):
        t.grad = torch.tensor(g.astype(np.float64))
        opt.step()
        m, v = orc.adamw_moments(m, v, g, (0.9, 0.999))
        p = orc.adamw_param(p, m, v, 1e-2, i + 1, (0.9, 0.999), 1e-8, 0.1)
    assert np.allclose(p, t.detach().numpy(), rtol=1e-5, atol=1e-7)


def test_swiglu_definition_against_differences():
    r = np.random.RandomState(2)
    g, u, dh, w = r.randn(5, 7), r.randn(5, 7), r.randn(5, 7), r.rand(5) + 0.5
    dg, du, dw = orc.swiglu_backward(g, u, dh, 0.6, w)
    f = lambda g, u, w: (dh * w[:, None] * orc.swiglu(g, u, 0.6)[3])  # noqa: E731
    e = 1e-6
    assert np.allclose((f(g + e, u, w) - f(g - e, u, w)) / (2 * e), dg, atol=1e-7)
    assert np.allclose((f(g, u + e, w) - f(g, u - e, w)) / (2 * e), du, atol=1e-7)
    assert np.allclose((f(g, u, w + e) - f(g, u, w - e)).sum(1) / (2 * e), dw, atol=1e-7)


def test_grouped_definitions_are_gradients_of_the_forward():
    """dgrad and wgrad against torch's autograd of a loop over the groups."""
    g = torch.Generator()
    g.manual_seed(3)
    counts, N, K = [2, 0, 3], 5, 4
    off = np.concatenate([[0], np.cumsum(counts)])
    x, w, dy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((6, K), (3, N, K), (5, N)))
    m = np.array([5, 0, 0, -1, 2])
    xp, wp = x.clone().requires_grad_(), w.clone().requires_grad_()
    loss = 0
    for p in range(5):
        e = int(np.searchsorted(off[1:], p, side="right"))
        if m[p] >= 0:
            loss = loss + (wp[e] @ xp[m[p]] * dy[p]).sum()
    loss.backward()
    dx, _ = orc.grouped_dgrad(dy.numpy(), w.numpy(), off, np.zeros((5, K)))
    gx = np.zeros((6, K))
    for p in range(5):
        if m[p] >= 0:
            gx[m[p]] += dx[p]
    assert np.allclose(gx, xp.grad.numpy())
    dw, _ = orc.grouped_wgrad(dy.numpy(), x.numpy(), off, np.zeros((3, N, K)), x_map=m)
    assert np.allclose(dw, wp.grad.numpy())


# ---- plans with empty tensors --------------------------------------------------------------------

def empty_tensor(i, **kw):
    """A tensor of no values, whose arrays have no address (an empty torch tensor's is NULL)."""
    return adamw_tensor(i, n=0, param=None, grad=None, exp_avg=None, exp_avg_sq=None, **kw)


@needs_lib
@pytest.mark.parametrize("empty_at", [(0,), (1,), (2,), (0, 1), (0, 2)], ids=str)
@pytest.mark.parametrize("master", [False, True])
def test_adamw_plan_takes_empty_tensors_anywhere(empty_at, master):
    """Whether the plan has master weights is said by the tensors that hold values."""
    ts = [empty_tensor(i) if i in empty_at else adamw_tensor(i, master=at(10 * i + 5) if master else None) for i in range(3)]
    rc, p, image = plan(ts)
    assert rc == 0, moe.load_library().moe_last_error()
    assert p.n_chunks == 3 - len(empty_at)
    flags = np.frombuffer(image, dtype=np.uint64, count=4)[3]
    assert flags == p.flags and bool(flags & 8) == master


@needs_lib
@pytest.mark.parametrize("tensors,kw,words", [
    (lambda: [empty_tensor(0, master=at(5)), adamw_tensor(1), adamw_tensor(2, master=at(25))], {}, b"tensor 2: master weights"),
    (lambda: [empty_tensor(0), adamw_tensor(1, master=at(15)), adamw_tensor(2)], {}, b"tensor 2: master weights"),
    (lambda: [empty_tensor(0), adamw_tensor(1, master=at(15))], dict(pd=1), b"belong to bf16 parameters"),
])
def test_adamw_plan_refuses_some_master_weights_behind_an_empty_tensor(tensors, kw, words):
    assert plan(tensors(), **kw)[0] == INVALID
    assert words in moe.load_library().moe_last_error()


@needs_lib
def test_adamw_plan_of_empty_tensors_only():
    rc, p, _ = plan([empty_tensor(0), empty_tensor(1)])
    assert rc == 0 and p.n_chunks == 0
    cfg = moe._AdamWConfig(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1)
    assert moe.load_library().moe_adamw_step(ctypes.byref(cfg), ctypes.byref(p), None, None) == 0


# ---- what an output may not overlap --------------------------------------------------------------

def swiglu_bwd_on(n=10, R=10, C=64, dgate=at(4), dup=at(5), row_w=at(6), pos=at(7), dw=at(8)):
    return moe.load_library().moe_swiglu_backward(n, R, C, 0.0, at(1), at(2), C, at(3), C, row_w, pos, dgate, dup, C, dw, None)


LAST = 10 * 64 * 2 - 4                     # the last four bytes of a [10, 64] bf16 matrix


@needs_lib
@pytest.mark.parametrize("call,words", [
    # the offsets and row maps of a product
    (lambda: forward(y=at(0)), b"y overlaps offsets"),
    (lambda: forward(groups(offsets=at(3) + 99 * 128 + 124)), b"y overlaps offsets"),
    (lambda: forward(x=rows(1, 128, row_map=at(3) + 16)), b"y overlaps row_map"),
    (lambda: forward(y=at(4) + 400 - 16, x=rows(1, 128, row_map=at(4))), b"y overlaps row_map"),
    (lambda: dgrad(dx=at(0) + 16), b"dx overlaps offsets"),
    (lambda: dgrad(dy=rows(1, 64, row_map=at(3))), b"dx overlaps row_map"),
    (lambda: wgrad(dw=at(0)), b"dw overlaps offsets"),
    (lambda: wgrad(dy=rows(1, 64, row_map=at(3) + 4 * 64 * 128 * 2 - 4)), b"dw overlaps the row map of dy"),
    (lambda: wgrad(x=rows(2, 128, row_map=at(3))), b"dw overlaps the row map of x"),
    # weights and positions of the activation
    (lambda: swiglu(w=at(3)), b"h overlaps row_w"),
    (lambda: swiglu(w=at(3) + LAST), b"h overlaps row_w"),
    (lambda: swiglu(pos=at(3) + 64), b"h overlaps pos"),
    (lambda: swiglu_bwd_on(dgate=at(6)), b"dgate overlaps row_w"),
    (lambda: swiglu_bwd_on(dup=at(6)), b"dup overlaps row_w"),
    (lambda: swiglu_bwd_on(dgate=at(7)), b"dgate overlaps pos"),
    (lambda: swiglu_bwd_on(dup=at(7)), b"dup overlaps pos"),
    (lambda: swiglu_bwd_on(dw=at(1) + LAST), b"drow_w overlaps gate"),
    (lambda: swiglu_bwd_on(dw=at(2)), b"drow_w overlaps up"),
    (lambda: swiglu_bwd_on(dw=at(3)), b"drow_w overlaps dh"),
    (lambda: swiglu_bwd_on(dw=at(4) + LAST), b"drow_w overlaps dgate"),
    (lambda: swiglu_bwd_on(dw=at(5)), b"drow_w overlaps dup"),
    (lambda: swiglu_bwd_on(dw=at(6) + 36), b"drow_w overlaps row_w"),
    (lambda: swiglu_bwd_on(dw=at(7)), b"drow_w overlaps pos"),
    (lambda: swiglu_bwd_on(R=0, dw=at(7)), b"drow_w overlaps pos"),
])
def test_overlap_refusals(call, words):
    assert call() == INVALID
    assert words in moe.load_library().moe_last_error()


# ---- arguments that are no tensors ---------------------------------------------------------------

F8 = torch.zeros(8)


@needs_lib
@pytest.mark.parametrize("wrong", [None, 3, [1.0, 2.0], np.zeros((4, 16), np.float32)], ids=["none", "number", "list", "array"])
@pytest.mark.parametrize("call,name", [
    (lambda t: moe.moe_grouped_gemm(t, bf(2, 8, 16), OFF, bf(4, 8)), "x"),
    (lambda t: moe.moe_grouped_gemm(bf(4, 16), t, OFF, bf(4, 8)), "w"),
    (lambda t: moe.moe_grouped_gemm(bf(4, 16), bf(2, 8, 16), t, bf(4, 8)), "offsets"),
    (lambda t: moe.moe_grouped_gemm(bf(4, 16), bf(2, 8, 16), OFF, t), "y"),
    (lambda t: moe.moe_grouped_gemm_dgrad(t, bf(2, 8, 16), OFF, bf(4, 16)), "dy"),
    (lambda t: moe.moe_grouped_gemm_dgrad(bf(4, 8), bf(2, 8, 16), OFF, t), "dx"),
    (lambda t: moe.moe_grouped_gemm_wgrad(t, bf(4, 16), OFF, bf(2, 8, 16)), "dy"),
    (lambda t: moe.moe_grouped_gemm_wgrad(bf(4, 8), t, OFF, bf(2, 8, 16)), "x"),
    (lambda t: moe.moe_grouped_gemm_wgrad(t, bf(4, 16), OFF, bf(2, 8, 16), dy_map=i32(0, 1, 2, 3)), "dy"),
    (lambda t: moe.moe_grouped_gemm_wgrad(bf(4, 8), bf(4, 16), OFF, t), "dw"),
    (lambda t: moe.moe_swiglu(t, bf(4, 8), bf(4, 8)), "gate"),
    (lambda t: moe.moe_swiglu(bf(4, 8), t, bf(4, 8)), "up"),
    (lambda t: moe.moe_swiglu(bf(4, 8), bf(4, 8), t), "h"),
    (lambda t: moe.moe_swiglu_backward(bf(4, 8), bf(4, 8), t, bf(4, 8), bf(4, 8)), "dh"),
    (lambda t: moe.moe_swiglu_backward(bf(4, 8), bf(4, 8), bf(4, 8), bf(4, 8), t), "dup"),
    (lambda t: moe.MoEAdamWPlan([t], [bf(8)], [F8], [F8]), "params[0]"),
    (lambda t: moe.MoEAdamWPlan([bf(8), bf(8)], [bf(8), t], [F8, F8], [F8, F8]), "grads[1]"),
    (lambda t: moe.MoEAdamWPlan([bf(8)], [bf(8)], [t], [F8]), "exp_avg[0]"),
    (lambda t: moe.MoEAdamWPlan([bf(8)], [bf(8)], [F8], [F8], master=[t]), "master[0]"),
    (lambda t: moe.moe_adamw_dequantise(t, F8, F8, True), "codes"),
    (lambda t: moe.moe_adamw_dequantise(u8(8), t, F8, True), "scales"),
    (lambda t: moe.moe_adamw_dequantise(u8(8), torch.zeros(1), t, True), "out"),
])
def test_binding_refuses_what_is_no_tensor(call, name, wrong):
    with pytest.raises(moe.MoEError) as e:
        call(wrong)
    assert e.value.status == INVALID and f"{name} must be a tensor" in str(e.value)


@needs_lib
@pytest.mark.parametrize("call,words", [
    (lambda: moe.moe_grouped_gemm(bf(4, 16), bf(2, 8, 16), OFF, bf(4, 8), row_map=[0, 1, 2, 3]), "the row map of x must be a tensor"),
    (lambda: moe.moe_grouped_gemm_wgrad(bf(4, 8), bf(4, 16), OFF, bf(2, 8, 16), x_map=[0, 1, 2, 3]), "the row map of x must be a tensor"),
    (lambda: moe.moe_grouped_gemm_dgrad(bf(4, 8), bf(2, 8, 16), OFF, bf(4, 16), dy2=[0], w2=bf(2, 8, 16)), "dy2 must be a tensor"),
    (lambda: moe.moe_grouped_gemm_dgrad(bf(4, 8), bf(2, 8, 16), OFF, bf(4, 16), dy2=bf(4, 8), w2=[0]), "w2 must be a tensor"),
    (lambda: moe.moe_grouped_gemm_wgrad(torch.tensor(1.0), bf(4, 16), OFF, bf(2, 8, 16)), "dy must have 2 dimension"),
    (lambda: moe.moe_grouped_gemm_wgrad(bf(4, 8), bf(4, 16), OFF, bf(2, 8, 16), x_map=torch.tensor(1)), "the row map of x must have 1 dimension"),
    (lambda: moe.moe_swiglu(bf(4, 8), bf(4, 8), bf(4, 8), pos=[0, 1]), "pos must be a tensor"),
    (lambda: moe.moe_swiglu(bf(4, 8), bf(4, 8), bf(4, 8), row_w=[0.5] * 4), "row_w must be a tensor"),
    (lambda: moe.moe_swiglu_backward(bf(4, 8), bf(4, 8), bf(4, 8), bf(4, 8), bf(4, 8), drow_w=[0.0] * 4), "drow_w must be a tensor"),
    (lambda: moe.MoEAdamWPlan([bf(8)], [bf(8)], [F8], [F8], weight_decay=[0.1, 0.2]), "weight_decay has 2 entries, params 1"),
    (lambda: moe.MoEAdamWPlan([bf(8)], [bf(8)], [F8], [F8], weight_decay=torch.tensor(0.1)), "one GPU must hold them all"),
    (lambda: moe.moe_adamw_step(None, lr=1e-3, step=1), "plan must be a MoEAdamWPlan"),
])
def test_binding_refuses_other_wrong_arguments(call, words):
    with pytest.raises(moe.MoEError) as e:
        call()
    assert e.value.status == INVALID and words in str(e.value)


# ---- the range of the 8-bit states ---------------------------------------------------------------

@pytest.mark.parametrize("ratio", [0.25, 0.99, 1.0, 1.03, 1.0625, 1.1, 1.125, 1.3, 2.0, 100.0])
@pytest.mark.parametrize("signed", [True, False])
def test_state_rounding_at_the_low_end(ratio, signed):
    """Read-back means of a value of `ratio` times the format's low end (2^-15 of the scale for the
    first moment, 2^-31 for the second).  First moment: zero up to 2^-15, rising to the value at
    1.125 2^-15 (the smallest code), unbiased from there.  Second: raised to 2^-31 below it, unbiased
    above.  A rounding has two outcomes, at most 1/8 of the lower one or (at the zero code) 1.125 2^-15
    apart, so N of them have a mean within 5 (apart / 2) / sqrt(N) of its expectation; the 16 random
    bits move the expectation by at most apart 2^-16, and fp32 rounds the value by 2^-22 of it."""
    low, N = 2.0 ** (-15 if signed else -31), 127 * 200
    value = ratio * low
    x = np.full(128, value, np.float32)
    x[0] = 1.875                                      # a scale of 1 (but for its rounding)
    got = np.mean([orc.state_decode(*orc.state_encode(x, signed, 0, s, 1), signed)[1:].astype(np.float64).mean() for s in range(200)])
    if signed:
        want = 0.0 if ratio <= 1 else min(9 * (ratio - 1) * low, value) if ratio < 1.125 else value
        apart = 0.0 if ratio < 1 else 1.125 * low if ratio < 1.125 else value / 8
    else:
        want, apart = max(value, low), 0.0 if ratio < 1 else value / 8
    # (at 2^-15 itself the rounding of the scale decides the side)
    assert abs(got - want) <= 5 * apart / 2 / N ** 0.5 + apart * 2.0 ** -16 + 9 * 2.0 ** -22 * value


@needs_lib
@pytest.mark.parametrize("call,words", [
    (lambda: moe.MoEAdamWPlan(None, [bf(8)], [F8], [F8]), "params must be a list of tensors"),
    (lambda: moe.MoEAdamWPlan([bf(8)], 7, [F8], [F8]), "grads must be a list of tensors"),
    (lambda: moe.MoEAdamWPlan([bf(8)], [bf(8)], torch.tensor(1.0), [F8]), "exp_avg must be a list of tensors"),
    (lambda: moe.MoEAdamWPlan([bf(8)], [bf(8)], [F8], [F8], master=1.5), "master must be a list of tensors"),
    (lambda: moe.MoEAdamWPlan([bf(8)], [bf(8)], [F8], [F8], weight_decay=None), "weight_decay must be a number"),
    (lambda: moe.MoEAdamWPlan([bf(8)], [bf(8)], [F8], [F8], weight_decay=[None]), "weight_decay must be a number"),
    (lambda: moe.MoEAdamWPlan([bf(8)], [bf(8)], [F8], [F8], weight_decay="fast"), "weight_decay must be a number"),
])
def test_adamw_plan_refuses_what_is_no_list(call, words):
    with pytest.raises(moe.MoEError) as e:
        call()
    assert e.value.status == INVALID and words in str(e.value)
