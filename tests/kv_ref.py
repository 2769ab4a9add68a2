"""Plain 64-bit forms of the rotary positions, the paged 8-bit cache and its
attention (numpy, loops over the definition), which the GPU tests compare with."""
import numpy as np

BLOCK = 16
_C = np.arange(256)
_E, _M = _C >> 3 & 15, _C & 7
E4M3 = np.where(_E > 0, (8 + _M) * 2.0 ** (_E - 10), _M * 2.0 ** -9) * np.where(_C > 127, -1.0, 1.0)
E4M3[[127, 255]] = np.nan


def rope(x, positions, freqs, style="half", amplitude=1.0, inverse=False):
    """[rows][heads][dim] in 64 bits."""
    x = np.asarray(x, np.float64)
    a = np.asarray(positions, np.float64)[:, None, None] * np.asarray(freqs, np.float64)
    a = -a if inverse else a
    amplitude = float(np.float32(amplitude))
    c, s = np.cos(a) * amplitude, np.sin(a) * amplitude
    n = len(freqs)
    y = x.copy()
    i0, i1 = (slice(0, n), slice(n, 2 * n)) if style == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    with np.errstate(invalid="ignore"):
        y[..., i0], y[..., i1] = x[..., i0] * c - x[..., i1] * s, x[..., i1] * c + x[..., i0] * s
    return y


def encode(v, code):
    """E4M3 codes of v / 2^(code - 127), nearest, ties to even; NaN and infinities: NaN."""
    v = np.asarray(v, np.float64)
    u = np.where(np.isfinite(v), v, 0.0) * 2.0 ** (127.0 - code)
    a = np.abs(u)
    e = np.clip(np.floor(np.log2(np.maximum(a, 1e-300))), -6, None)
    # (log2 of a number just below a power of two may round up to it)
    e = np.where(2.0 ** e > a, np.maximum(e - 1, -6), e)
    n = np.rint(a / 2.0 ** (e - 3))  # eighths of the leading power: 8 .. 16, below 8 for subnormals
    up = n == 16
    e, n = np.where(up, e + 1, e), np.where(up, 8, n)
    q = np.where(n < 8, n, (e + 7) * 8 + n - 8).astype(np.int64)
    assert (q <= 126).all()
    q = np.where(np.signbit(u), q + 128, q)
    return q.astype(np.uint8), ~np.isfinite(v)


def scale_code(amax):
    if amax == 0:
        return 0
    m, e = np.frexp(amax)
    return max(int(e) - 9 + int(m > 0.875) + 127, 0)


class Cache:
    """kv uint8 [2][pages][heads][page][dim], scale uint8 [2][pages][heads][page/16]."""

    def __init__(self, kv, scale, table):
        self.kv, self.scale, self.table = kv.copy(), scale.copy(), table
        _, self.pages, self.heads, self.page, self.dim = kv.shape

    def _at(self, b, p):
        """(page, slot) of a position, or None."""
        if p < 0 or p >= self.table.shape[1] * self.page:
            return None
        pg = int(self.table[b, p // self.page])
        return (pg, p % self.page) if 0 <= pg < self.pages else None

    def append(self, k, v, starts, lens, freqs=None, style="half", amplitude=1.0):
        """k, v [rows][heads][dim] as float64 of BF16 values."""
        for b in range(len(lens)):
            n = starts[b + 1] - starts[b]
            blocks = {}
            for i in range(n):
                p = int(lens[b]) - n + i
                if self._at(b, p) is not None:
                    blocks.setdefault(p // BLOCK, []).append((p, starts[b] + i))
            for blk, rows in blocks.items():
                pg, _ = self._at(b, blk * BLOCK)
                at = [p % self.page for p, _ in rows]
                i = [r for _, r in rows]
                kk = k[i] if freqs is None else rope(k[i], [p for p, _ in rows], freqs, style, amplitude)
                x = np.stack([kk, v[i]])
                with np.errstate(over="ignore"):
                    x = np.where(np.isinf(x.astype(np.float32)), np.copysign(np.inf, x), x)  # beyond FP32's range
                s = at[0] // BLOCK
                off = at[0] % BLOCK
                for w in range(2):
                    for h in range(self.heads):
                        fin = x[w, :, h][np.isfinite(x[w, :, h])]
                        c = scale_code(np.abs(fin).max() if fin.size else 0.0)
                        old = int(self.scale[w, pg, h, s])
                        if off > 0 and old < c:
                            cells = self.kv[w, pg, h, s * BLOCK:s * BLOCK + off]
                            was = E4M3[cells] * 2.0 ** (old - 127.0)
                            q, bad = encode(was, c)
                            cells[:] = np.where(bad, 0x7F, q)
                        elif off > 0:
                            c = old
                        q, bad = encode(x[w, :, h], c)
                        self.kv[w, pg, h, at] = np.where(bad, 0x7F, q)
                        self.scale[w, pg, h, s] = c

    def row(self, b, p):
        """Values [2][heads][dim] of a position, or None."""
        at = self._at(b, p)
        if at is None:
            return None
        pg, slot = at
        c = self.scale[:, pg, :, slot // BLOCK].astype(np.float64)
        with np.errstate(invalid="ignore"):
            return np.where(c == 255, np.nan, 2.0 ** (c - 127.0))[..., None] * E4M3[self.kv[:, pg, :, slot]]

    def read(self, starts, lens, rows):
        out = np.full((2, rows, self.heads, self.dim), np.nan)
        for b in range(len(lens)):
            n = starts[b + 1] - starts[b]
            for i in range(n):
                v = self.row(b, int(lens[b]) - n + i)
                out[:, starts[b] + i] = 0.0 if v is None else v
        return out

    def attention(self, q, starts, lens, scale, causal=True, window=0):
        """(out, lse, w): out and lse in 64 bits, w the bound's ingredients of every (row, head):
        sum of weights times |v| [dim], and the largest sum of |q k| * scale."""
        rows, heads, dim = q.shape
        g = heads // self.heads
        out, lse = np.full(q.shape, np.nan), np.full((rows, heads), np.nan)
        mag, reach = np.zeros(q.shape), np.zeros((rows, heads))
        for b in range(len(lens)):
            n = starts[b + 1] - starts[b]
            cells = [self.row(b, p) for p in range(min(max(int(lens[b]), 0), self.table.shape[1] * self.page))] if n else []
            for i in range(n):
                t, p = starts[b] + i, int(lens[b]) - n + i
                last = min(p, len(cells) - 1) if causal else len(cells) - 1
                first = max(p - window + 1, 0) if window else 0
                see = [j for j in range(first, last + 1) if cells[j] is not None]
                if not see:
                    out[t], lse[t] = 0.0, -np.inf
                    continue
                kv = np.stack([cells[j] for j in see], 1)  # [2][seen][heads][dim]
                for h in range(heads):
                    kk, vv = kv[0, :, h // g], kv[1, :, h // g]
                    s = kk @ q[t, h] * scale
                    m = s.max()
                    e = np.exp(s - m)
                    lse[t, h] = m + np.log(e.sum())
                    out[t, h] = e @ vv / e.sum()
                    mag[t, h] = e @ np.abs(vv) / e.sum()
                    reach[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * scale
        return out, lse, mag, reach
