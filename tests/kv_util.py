"""Caches and batches for the GPU tests of the paged 8-bit cache."""
import numpy as np
import torch

import kv_ref as ref

BF = torch.bfloat16


def bf16(rng, *shape, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(BF)


class Batch:
    """Sequences of new[b] rows behind ctx[b] positions, pages dealt out of order, the rest
    of the table -1 (room: positions that it has places for at least).  Cells that no
    position holds are filled with any bytes, NaN codes and scales among them."""

    def __init__(self, seed, new, ctx, heads, dim, page, layout="hnd", spare=2, behind=0, filled=True, std=1.0, room=0):
        self.rng = rng = np.random.default_rng(seed)
        self.new, self.ctx, self.heads, self.dim, self.page = list(new), list(ctx), heads, dim, page
        lens = [n + c for n, c in zip(new, ctx)]
        need = [max(0, -(-n // page)) for n in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        self.table = np.full((len(new), max(max(need + [1]) + 1, -(-room // page))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lens = np.array(lens, np.int32)
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.rows = int(self.starts[-1]) + behind
        kv = rng.integers(0, 256, (2, pages, heads, page, dim)).astype(np.uint8)
        scale = rng.integers(0, 256, (2, pages, heads, page // 16)).astype(np.uint8)
        if filled:
            for b, c in enumerate(lens):
                for p in range(c):
                    pg, slot = self.table[b, p // page], p % page
                    if slot % 16 == 0:
                        scale[:, pg, :, slot // 16] = rng.integers(117, 122, (2, heads))
                    x = rng.standard_normal((2, heads, dim)) * std
                    for w in range(2):
                        for h in range(heads):
                            code = int(scale[w, pg, h, slot // 16])
                            kv[w, pg, h, slot], _ = ref.encode(np.clip(x[w, h], -448 * 2.0 ** (code - 127), 448 * 2.0 ** (code - 127)), code)
        self.ref = ref.Cache(kv, scale, self.table)
        t = torch.from_numpy(kv).cuda()
        if layout == "nhd":  # [2][pages][page][heads][dim] in memory
            t = t.transpose(2, 3).contiguous().transpose(2, 3)
        elif layout == "alternate":  # keys and values of a page together
            t = t.transpose(0, 1).contiguous().transpose(0, 1)
        elif layout == "padded":
            wide = torch.zeros(2, pages, heads, page + 3, dim + 16, dtype=torch.uint8, device="cuda")
            wide[:, :, :, :page, :dim] = t
            t = wide[:, :, :, :page, :dim]
        self.kv, self.scale = t, torch.from_numpy(scale).cuda()

    @property
    def args(self):
        """The cache's and the batch's arguments after the data."""
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        return self.kv, self.scale, dev(self.table), dev(self.lens), dev(self.starts)

    def kv_np(self):
        return self.kv.cpu().numpy()

    def scale_np(self):
        return self.scale.cpu().numpy()


def attention_bounds(want, lse, mag, reach, dim, keys):
    """Allowed errors of (out, lse).

    A score is a sum of dim exact products in FP32 (dim half steps of the sum of their
    magnitudes, twice that for truncating adders) and three roundings of its scaling; with e the
    bound of a score's error, a weight's is 2 e + 8 * 2^-24 (difference from the maximum, exp2, rescaling),
    its rounding to BF16 2^-8, the sums' keys * 2^-24; the normalizer has the same without BF16."""
    e = (2 * dim + 8) * 2.0 ** -24 * reach
    rel = 4 * e + (16 + 2 * keys) * 2.0 ** -24
    out = (2.0 ** -8 + rel[..., None]) * mag + 2.0 ** -8 * np.abs(want) + 1e-37
    with np.errstate(invalid="ignore"):
        lo = 2 * e + (16 + keys) * 2.0 ** -24 + np.where(np.isfinite(lse), np.abs(lse), 0) * 4 * 2.0 ** -24
    return out, lo


def check_attention(got, got_lse, ref_result, dim, keys):
    want, lse, mag, reach = ref_result
    out = got.double().cpu().numpy()
    ob, lb = attention_bounds(want, lse, mag, reach, dim, keys)
    nan = np.isnan(want)
    assert (np.isnan(out) == nan).all(), "NaN in other places"
    err = np.where(nan, 0, np.abs(out - np.where(nan, 0, want)))
    ok = err <= np.where(nan, 1, ob)
    assert ok.all(), (np.argwhere(~ok)[:4], (err / np.where(nan, 1, ob)).max())
    if got_lse is not None:
        g = got_lse.double().cpu().numpy()
        same = (np.isnan(g) == np.isnan(lse)) & (np.isneginf(g) == np.isneginf(lse))
        assert same.all(), np.argwhere(~same)[:4]
        fin = np.isfinite(lse)
        err = np.abs(g[fin] - lse[fin])
        assert (err <= lb[fin]).all(), (err / lb[fin]).max()
