"""fp64 oracle of the low-rank adapter products, their gradients and the 8-bit
activations (include/gptq.h, gptq_lora_* and gptq_*_act8), in NumPy.

The magnitudes (``mag`` and the like) are the same sums over absolute values,
which the tests' error bounds are stated in.
"""
import numpy as np


def plan(ids, slots):
    """(order, slot_start): tokens by slot, in token order within a slot;
    ids below 0 or from ``slots`` on have no slot and come last."""
    ids = np.asarray(ids)
    key = np.where((ids < 0) | (ids >= slots), slots, ids)
    order = np.argsort(key, kind="stable")
    start = np.searchsorted(key[order], np.arange(slots + 1))
    return order.astype(np.int32), start.astype(np.int32)


def _slots(A, ids, ranks):
    for a in range(A.shape[0]):
        r = A.shape[1] if ranks is None else int(min(max(ranks[a], 0), A.shape[1]))
        t = np.nonzero(np.asarray(ids) == a)[0]
        if t.size and r:
            yield a, r, t


def project(x, A, ids, ranks=None):
    """u (ntok, max_rank): x A^T of each token's adapter; NaN rows where a
    token has none (they are not written)."""
    S, rmax, _ = A.shape
    ids = np.asarray(ids)
    u = np.full((x.shape[0], rmax), np.nan)
    u[(ids >= 0) & (ids < S)] = 0.0
    for a, r, t in _slots(A, ids, ranks):
        u[t, :r] = x[t] @ A[a, :r].T
    return u


def apply(x, A, B, ids, ranks, scales, y):
    """(y + delta, u, magnitude of u, magnitude of delta)."""
    out, dmag = y.copy(), np.zeros_like(y)
    u = project(x, A, ids, ranks)
    umag = project(np.abs(x), np.abs(A), ids, ranks)
    for a, r, t in _slots(A, ids, ranks):
        s = 1.0 if scales is None else float(scales[a])
        out[t] += s * (u[t, :r] @ B[a, :, :r].T)
        dmag[t] = abs(s) * (umag[t, :r] @ np.abs(B[a, :, :r]).T)
    return out, u, umag, dmag


def backward(dy, u, x, A, B, ids, ranks, scales, dx):
    """dict of dx, dA, dB and of their magnitudes mdx, mdA, mdB (of what the
    adapters add, over absolute values)."""
    S, rmax, n = A.shape
    m = B.shape[1]
    o = {"dx": dx.copy(), "mdx": np.zeros_like(dx), "dA": np.zeros((S, rmax, n)),
         "mdA": np.zeros((S, rmax, n)), "dB": np.zeros((S, m, rmax)),
         "mdB": np.zeros((S, m, rmax))}
    for a, r, t in _slots(A, ids, ranks):
        s = 1.0 if scales is None else float(scales[a])
        Aa, Ba = A[a, :r], B[a, :, :r]
        v, vm = s * (dy[t] @ Ba), abs(s) * (np.abs(dy[t]) @ np.abs(Ba))
        o["dx"][t] += v @ Aa
        o["mdx"][t] = vm @ np.abs(Aa)
        o["dA"][a, :r] = v.T @ x[t]
        o["mdA"][a, :r] = vm.T @ np.abs(x[t])
        o["dB"][a, :, :r] = s * (dy[t].T @ u[t, :r])
        o["mdB"][a, :, :r] = abs(s) * (np.abs(dy[t]).T @ np.abs(u[t, :r]))
    return o


def quantize_act8(x, group):
    """(codes, scales fp32) of x (rows, n), float64 holding bf16 or fp32
    values: the scale is rounded to fp32 once, the quotient is not rounded
    before it is turned into a code (float64 separates every quotient of two
    fp32 values that is not a tie from the tie next to it)."""
    rows, n = x.shape
    g = n if group < 0 else group
    G = (n + g - 1) // g
    codes = np.zeros((rows, n), np.int8)
    scales = np.zeros((rows, G), np.float32)
    for k in range(G):
        w = x[:, k * g:(k + 1) * g]
        fine = np.isfinite(w).all(axis=1)
        amax = np.where(fine, np.abs(np.where(np.isfinite(w), w, 0.0)).max(axis=1), 0.0)
        sc = np.maximum((amax / 127.0).astype(np.float32), np.float32(2.0 ** -126))
        q = np.rint(np.where(fine[:, None], w, 0.0) / sc.astype(np.float64)[:, None])
        codes[:, k * g:(k + 1) * g] = np.clip(q, -127, 127).astype(np.int8)
        scales[:, k] = np.where(fine, sc, np.float32(np.nan))
    return codes, scales


def dequant_act8(codes, scales, group):
    """The fp32 values (one rounded multiply) that the codes stand for."""
    n = codes.shape[1]
    g = n if group < 0 else group
    sc = np.repeat(scales.astype(np.float32), g, axis=1)[:, :n]
    return sc * codes.astype(np.float32)
