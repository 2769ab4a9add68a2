"""Plain 64-bit reference of the routing, its gradients and MXFP4 (numpy, CPU).

MXFP4 rule (OCP Microscaling Formats v1.0): per 32 elements amax = max |v|,
scale code c = floor(log2 amax) - 2 + 127 clamped to [0, 254]; elements
v / 2^(c-127) to the nearest E2M1 value, ties to the even code, above 6
clamped; a block with NaN or Inf: c = 0xFF, codes 7; a zero block: c = 0.
"""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def bf16_values(bits: np.ndarray) -> np.ndarray:
    with np.errstate(invalid="ignore"):   # NaN patterns
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantize(bits: np.ndarray):
    """BF16 patterns [rows][cols] -> (codes [rows][cols], scales [rows][cols/32])."""
    rows, cols = bits.shape
    v = bf16_values(bits).reshape(rows, -1, 32)
    bad = ~np.isfinite(v).all(-1)
    a = np.where(bad[..., None], 1.0, np.abs(v))
    amax = a.max(-1)
    _, e = np.frexp(np.where(amax > 0, amax, 1.0))
    c = np.where(amax > 0, np.clip(e - 1 - 2 + 127, 0, 254), 0)
    x = np.ldexp(a, (127 - c)[..., None].astype(int))
    lo = np.clip(np.searchsorted(E2M1, x, side="right") - 1, 0, 7)
    hi = np.minimum(lo + 1, 7)
    below, above = x - E2M1[lo], E2M1[hi] - x
    code = np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)
    code = np.where(x >= 6, 7, code)
    sign = ((bits.reshape(v.shape) >> 15) & 1).astype(int)
    code = np.where(bad[..., None], 7, code | (sign << 3))
    return code.reshape(rows, cols).astype(np.uint8), np.where(bad, 0xFF, c).astype(np.uint8)


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(q: np.ndarray) -> np.ndarray:
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    s = np.where(scales == 0xFF, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return v * np.repeat(s, 32, axis=1)


def route(x, topk, softmax, bias=None, groups=1, keep=1, group_top=1, renorm=True, scale=1.0, mask=None):
    """(ids, weights) by the definition, row by row."""
    T, E = x.shape
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        r = x[t].astype(np.float64)
        with np.errstate(all="ignore"):
            s = np.exp(r - r.max()) / np.exp(r - r.max()).sum() if softmax else 1 / (1 + np.exp(-r))
        key = r if bias is None and group_top == 1 else s + (0 if bias is None else bias.astype(np.float64))
        key = np.where(r == -np.inf, -np.inf, key)
        key = np.where(np.isnan(key), np.inf, key)    # ranks first
        if groups > 1:
            by = key.reshape(groups, -1)
            best = -np.sort(-by, axis=1)[:, :group_top].sum(1)
            chosen = np.argsort(-best, kind="stable")[:keep]
            live = np.zeros(groups, bool)
            live[chosen] = True
            key = np.where(np.repeat(live, E // groups), key, -np.inf)
        order = np.argsort(-key, kind="stable")[:topk]
        order = order[key[order] > -np.inf]
        ids[t, :len(order)] = order
        if renorm:
            z = r[order]
            if softmax:
                q = np.exp(z - z.max()) if len(z) else z
            else:
                ls = -np.logaddexp(0, -z)
                q = np.exp(ls - ls.max()) if len(z) else z
            w[t, :len(order)] = scale * q / q.sum() if len(z) else 0
        else:
            w[t, :len(order)] = scale * s[order]
    return ids, w


def route_bwd(x, ids, g, softmax, renorm=True, scale=1.0):
    """Gradient of sum g * weights with respect to x (64 bits), ids fixed."""
    T, E = x.shape
    dx = np.zeros((T, E))
    for t in range(T):
        r = x[t].astype(np.float64)
        ok = np.array([0 <= i < E and r[i] > -np.inf for i in ids[t]], bool)
        sel, gt = ids[t][ok], g[t][ok].astype(np.float64)
        if not len(sel):
            continue
        s = np.exp(r - r.max()) / np.exp(r - r.max()).sum() if softmax else 1 / (1 + np.exp(-r))
        if renorm:
            S = s[sel].sum()
            ds = scale * (gt - (gt * s[sel]).sum() / S) / S
        else:
            ds = scale * gt
        dense = np.zeros(E)
        np.add.at(dense, sel, ds)
        dx[t] = s * (dense - (dense * s).sum()) if softmax else dense * s * (1 - s)
    return dx
