"""Float64 definitions of the operators that train the router (NumPy, test infrastructure): the balance
loss of sequences, and the gradient of the logits through the mixing weights and through that loss."""
from collections import namedtuple

import numpy as np

Balance = namedtuple("Balance", "counts probs loss")
Backward = namedtuple("Backward", "dlogits dlogits_mag")


def _sigmoid(l):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-l))


def runs(T, offsets=None, lens=None):
    """(begin, end) of every sequence's tokens, arrays taken as the kernels take them."""
    out = []
    for b in range(1 if offsets is None else len(offsets) - 1):
        lo, hi = 0, T
        if offsets is not None:
            lo = min(max(offsets[b], 0), T)
            hi = min(max(offsets[b + 1], lo), T)
        out.append((lo, hi if lens is None else lo + min(max(lens[b], 0), hi - lo)))
    return out


def _shares(s):
    total = s.sum(1, keepdims=True)
    return np.divide(s, total, out=np.zeros_like(s), where=total != 0)


def balance_loss(logits, idx, K, coef, offsets=None, lens=None):
    T, E = logits.shape
    rs = runs(T, offsets, lens)
    N = sum(hi - lo for lo, hi in rs)
    p = _shares(_sigmoid(logits))
    counts, probs, loss = np.zeros((len(rs), E), np.int32), np.zeros((len(rs), E)), 0.0
    for b, (lo, hi) in enumerate(rs):
        if hi <= lo:
            continue
        ids = idx[lo:hi].reshape(-1)
        counts[b] = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        probs[b] = p[lo:hi].mean(0)
        loss += (hi - lo) / N * (E * counts[b] / (K * (hi - lo)) * probs[b]).sum()
    return Balance(counts, probs, coef * loss)


def router_backward(logits, idx, K, norm, scale, dtopk_w=None, counts=None, balance=0.0, offsets=None, lens=None):
    """dlogits and the sum of the magnitudes of its terms; balance = dloss * coef."""
    T, E = logits.shape
    s = _sigmoid(logits)
    r = _sigmoid(-logits)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    if counts is not None:
        p, rs = _shares(s), runs(T, offsets, lens)
        N = sum(hi - lo for lo, hi in rs)
        for b, (lo, hi) in enumerate(rs):
            if hi <= lo:
                continue
            f, q = E * counts[b] / (K * (hi - lo)), p[lo:hi]
            d[lo:hi] = balance / N * (f - (q @ f)[:, None]) * q * r[lo:hi]
            mag[lo:hi] = abs(balance) / N * (f + (q @ f)[:, None]) * q * r[lo:hi]
    if dtopk_w is not None:
        for t in range(T):
            ok = (idx[t] >= 0) & (idx[t] < E)
            e, g = idx[t][ok], dtopk_w[t][ok] * scale
            sk = s[t, e]
            if norm:
                q = sk / sk.sum() if sk.sum() else sk
                v, m = (g - (g * q).sum()) * q * r[t, e], (np.abs(g) + (np.abs(g) * q).sum()) * q * r[t, e]
            else:
                v = g * sk * r[t, e]
                m = np.abs(v)
            np.add.at(d[t], e, v)
            np.add.at(mag[t], e, m)
    return Backward(d, mag)
