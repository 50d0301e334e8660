"""The norm in front of the layer and the router's training side, in float64.

Plain numpy from the definitions, one function per operator.  Inputs are
float64 arrays holding the values of whatever type the operator reads; where
the operator rounds (the residual sum, the 8-bit output), the rounding is made
here on the values.
"""
import numpy as np


def round_bf16(v):
    """float32 values rounded to bf16 (half to even), as float32."""
    u = np.asarray(v, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    return np.where(np.isnan(v), np.float32(np.nan), (r & 0xFFFFFFFF).astype(np.uint32).view(np.float32))


def e4m3_values():
    """The values of the e4m3 codes 0 .. 126 (127 is NaN), increasing."""
    c = np.arange(127)
    ex, man = c >> 3, c & 7
    return np.where(ex == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (ex - 10.0))


def mx8_encode(v):
    """(codes uint8 [T][H], scales uint8 [T][H/32]) of float64 rows."""
    T, H = v.shape
    table = e4m3_values()
    b = v.reshape(T, H // 32, 32)
    finite = np.isfinite(b).all(axis=2)
    mag = np.where(finite[:, :, None], np.abs(b), 0.0)
    amax = mag.max(axis=2) if H else np.zeros((T, 0))
    grid = 448.0 * 2.0 ** np.arange(-127, 128)
    s = np.minimum(np.searchsorted(grid, amax), 254)           # least e + 127 with amax <= 448 2^e
    u = mag / 2.0 ** (s[:, :, None] - 127.0)
    hi = np.clip(np.searchsorted(table, u), 1, 126)
    lo = hi - 1
    dl, dh = u - table[lo], table[hi] - u
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code | np.where(np.signbit(b), 0x80, 0)
    code = np.where(finite[:, :, None], code, 0x7F).astype(np.uint8)
    return code.reshape(T, H), np.where(finite, s, 255).astype(np.uint8)


def mx8_decode(codes, scales):
    table = np.concatenate([e4m3_values(), [np.nan]])
    v = table[codes & 0x7F] * np.where(codes & 0x80, -1.0, 1.0)
    sc = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(sc, 32, axis=1)


def rms_norm(x, residual, weight, eps, res_bf16, round_h):
    """h (float64 holding the stored values), r, n = h r, y = n weight."""
    h = np.asarray(x, dtype=np.float32)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float32)
    if round_h and res_bf16:
        h = round_bf16(h)
    h = h.astype(np.float64)
    r = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    n = h * r[:, None]
    return h, r, n, n * weight


def rms_norm_backward(dy, dres, n, r, weight, mask=None):
    """(dx, dweight); a masked token has no part and a zero row."""
    keep = np.ones(len(dy), bool) if mask is None else np.asarray(mask, bool)
    dx = np.zeros(dy.shape)
    g = dy[keep] * weight
    nk = n[keep]
    m = (g * nk).mean(axis=1, keepdims=True)
    dx[keep] = r[keep, None] * (g - nk * m) + (0.0 if dres is None else dres[keep])
    return dx, (dy[keep] * nk).sum(axis=0)


def softmax(z):
    """Row softmax; -inf gives 0, also in a row of nothing else."""
    m = z.max(axis=1, keepdims=True)
    p = np.exp(z - np.where(np.isneginf(m), 0.0, m))
    s = p.sum(axis=1, keepdims=True)
    return np.divide(p, s, out=np.zeros_like(p), where=s != 0)


def _members(T, mask, offsets):
    off = [0, T] if offsets is None else list(offsets)
    keep = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    return [[t for t in range(max(0, off[g]), min(T, off[g + 1])) if keep[t]] for g in range(len(off) - 1)]


def balance_loss(z, ids, E, k, alpha, mask=None, offsets=None):
    """dict of loss, counts, n_valid, prob_mean, and dlogits for dloss = 1."""
    groups = _members(len(z), mask, offsets)
    S = len(groups)
    live = sum(len(g) > 0 for g in groups)
    counts, mean, dz = np.zeros((S, E), np.int32), np.zeros((S, E)), np.zeros((len(z), E))
    loss = 0.0
    for g, rows in enumerate(groups):
        if not rows:
            continue
        n = len(rows)
        for e in ids[rows].reshape(-1):
            if 0 <= e < E:
                counts[g, e] += 1
        p = softmax(z[rows])
        mean[g] = p.sum(axis=0) / n
        f = counts[g] * (E / (k * n))
        loss += alpha / live * (f * mean[g]).sum()
        a = alpha / live * f / n
        dz[rows] = p * (a - (p * a).sum(axis=1, keepdims=True))
    return {"loss": loss, "counts": counts, "n_valid": np.array([len(g) for g in groups] + [live], np.int32),
            "prob_mean": mean, "dlogits": dz}


def route_dlogits(z, ids, w, dw, renormalize, dz_in, E, mask=None):
    """Gradient of the logits; ids outside [0, E) pass none."""
    T = len(ids) if ids is not None else len(dz_in)
    dz = np.zeros((T, E))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        if dw is not None:
            ok = (ids[t] >= 0) & (ids[t] < E)
            d = np.where(ok, dw[t], 0.0)
            dot = (w[t] * d)[ok].sum()
            if renormalize:
                for j in np.nonzero(ok)[0]:
                    dz[t, ids[t, j]] += w[t, j] * (d[j] - dot)
            else:
                p = softmax(np.where(np.isnan(z[t:t + 1]), -np.inf, z[t:t + 1]))[0]
                g = np.full(E, -dot)
                for j in np.nonzero(ok)[0]:
                    g[ids[t, j]] += d[j]
                dz[t] = p * g
        if dz_in is not None:
            dz[t] += dz_in[t]
    return dz


def route_backward(dz, x, w_router, mask=None):
    """(dx, dw_router, dbias) from the logits' gradient."""
    keep = slice(None) if mask is None else np.asarray(mask, bool)
    return dz @ w_router, dz[keep].T @ x[keep], dz.sum(axis=0)
