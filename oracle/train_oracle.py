"""Float64 definitions of the operators that train a layer's experts (NumPy, test infrastructure):
products grouped by expert, SwiGLU with clamp and routing weight, and the AdamW step, whose 8-bit
states are defined in fp32 operation by operation."""
import numpy as np

STATE_BLOCK, STATE_TOP = 128, np.float32(1.0 / 1.875)


def _rows(a, row_map, p):
    """Rows of positions p in float64; a row outside the matrix is zeros."""
    r = p if row_map is None else np.asarray(row_map)[p]
    ok = (r >= 0) & (r < a.shape[0])
    out = np.zeros((len(p), a.shape[1]))
    out[ok] = a[r[ok]]
    return out, ok


def grouped_forward(x, w, offsets, y, row_map=None, accumulate=False):
    """(result, sum of magnitudes) of y[p] = w[g] x[row_map[p]]; rows of no group keep y."""
    out, mag = np.array(y, dtype=np.float64), np.zeros(y.shape)
    for g in range(w.shape[0]):
        p = np.arange(offsets[g], offsets[g + 1])
        xr, _ = _rows(x, row_map, p)
        out[p] = xr @ w[g].T + (out[p] if accumulate else 0)
        mag[p] = np.abs(xr) @ np.abs(w[g]).T + (np.abs(y[p]) if accumulate else 0)
    return out, mag


def grouped_dgrad(dy, w, offsets, dx, row_map=None, dy2=None, w2=None, accumulate=False):
    wt = np.swapaxes(w, 1, 2)
    out, mag = grouped_forward(dy, wt, offsets, dx, row_map, accumulate)
    if dy2 is not None:
        out, m2 = grouped_forward(dy2, np.swapaxes(w2, 1, 2), offsets, out, row_map, True)
        lo, hi = offsets[0], offsets[-1]
        mag[lo:hi] += grouped_forward(dy2, np.swapaxes(w2, 1, 2), offsets, np.zeros_like(out), row_map)[1][lo:hi]
    return out, mag


def grouped_wgrad(dy, x, offsets, dw, dy_map=None, x_map=None, accumulate=False):
    out, mag = np.zeros(dw.shape), np.zeros(dw.shape)
    for g in range(dw.shape[0]):
        p = np.arange(offsets[g], offsets[g + 1])
        d, okd = _rows(dy, dy_map, p)
        r, okx = _rows(x, x_map, p)
        ok = okd & okx
        out[g] = d[ok].T @ r[ok]
        mag[g] = np.abs(d[ok]).T @ np.abs(r[ok])
    return (out + dw, mag + np.abs(dw)) if accumulate else (out, mag)


def swiglu(gate, up, limit):
    """(sigmoid, silu(gate) * up, whether the clamp leaves it, clamped) in float64."""
    with np.errstate(over="ignore"):
        sig = 1.0 / (1.0 + np.exp(-gate))
    a = gate * sig * up
    if not limit > 0:
        return sig, a, np.ones(a.shape, bool), a
    return sig, a, ~(np.abs(a) > limit), np.clip(a, -limit, limit)


def swiglu_backward(gate, up, dh, limit, row_w):
    """(dgate, dup, drow_w) for rows in the order of row_w."""
    sig, _, free, s = swiglu(gate, up, limit)
    da = dh * row_w[:, None] * free
    return da * up * sig * (1 + gate * (1 - sig)), da * gate * sig, (dh * s).sum(1)


# ---- AdamW ---------------------------------------------------------------------------------------

def adamw_moments(m, v, g, betas):
    """The new moments in fp32, each operation rounded by itself."""
    f = np.float32
    b1, o1, b2, o2 = f(betas[0]), f(1 - betas[0]), f(betas[1]), f(1 - betas[1])
    m, v, g = (np.asarray(t, dtype=f) for t in (m, v, g))
    return m * b1 + g * o1, v * b2 + (g * g) * o2


def adamw_param(p, m, v, lr, step, betas, eps, weight_decay):
    """The new parameter in float64 from the new moments."""
    m, v, p = (np.asarray(t, dtype=np.float64) for t in (m, v, p))
    mh, vh = m / (1 - betas[0] ** step), v / (1 - betas[1] ** step)
    return p * (1 - lr * weight_decay) - lr * mh / (np.sqrt(vh) + eps)


def state_bits16(n, tensor, seed, step):
    """16 random bits of each of a tensor's n values."""
    M = np.uint64(0xFFFFFFFF)
    pair = np.arange((n + 1) // 2, dtype=np.uint64) & M
    key = np.uint64((tensor * 0x9E3779B9 + seed + step * 0x7F4A7C15) & 0xFFFFFFFF)
    x = (pair * np.uint64(0x8DA6B343) + key) & M
    x ^= x >> np.uint64(15)
    x = (x * np.uint64(0xD8163841)) & M
    x ^= x >> np.uint64(13)
    x = (x * np.uint64(0xCB1AB31F)) & M
    x ^= x >> np.uint64(16)
    return np.stack([x & np.uint64(0xFFFF), x >> np.uint64(16)], 1).reshape(-1)[:n].astype(np.int64)


def state_encode(x, signed, tensor, seed, step):
    """fp32 values of one tensor -> (codes uint8, scales fp32)."""
    f, n = np.float32, len(x)
    nb = -(-n // STATE_BLOCK)
    pad = np.zeros(nb * STATE_BLOCK, f)
    pad[:n] = x
    with np.errstate(divide="ignore", invalid="ignore", over="ignore", under="ignore"):
        scale = np.abs(pad).reshape(nb, STATE_BLOCK).max(1) * STATE_TOP
        scale = np.where(scale < f(2.0 ** -126), f(0), scale).astype(f)
        inv = np.where(scale > 0, f(1) / scale, f(0)).astype(f)
        y = np.abs(pad) * np.repeat(inv, STATE_BLOCK)
    bits = y.view(np.int32).astype(np.int64)[:n] + (state_bits16(n, tensor, seed, step) << 4)
    code = np.clip((bits >> 20) - ((127 - (15 if signed else 31)) << 3), 0, 127 if signed else 255)
    if signed:
        code |= np.signbit(x).astype(np.int64) << 7
    return code.astype(np.uint8), scale


def state_decode(codes, scales, signed):
    c = codes.astype(np.int32)
    mag = c & 127 if signed else c
    y = ((mag << 20) + ((127 - (15 if signed else 31)) << 23)).astype(np.int32).view(np.float32)
    if signed:
        y = np.where(mag == 0, np.float32(0), np.where(c > 127, -y, y))
    with np.errstate(invalid="ignore"):
        return y * np.repeat(scales, STATE_BLOCK)[:len(codes)]
