"""The attention where its work is cut as real batches are: prompts of many steps whose tiles store their rows themselves
or join a few ranges, lines of chunks whose pieces end one item and start the next.  Each test says by the sizes that it
is there.  Reference: the definition in 64 bits on the device's codes, a head at a time; tolerances: tests/kv_util.py."""
import numpy as np
import pytest
import torch

import kv_ref as ref
from kv_util import BF, Batch, bf16, check_attention

pytestmark = pytest.mark.gpu

TABLE = torch.from_numpy(ref.E4M3)


def _units():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _ranges(B, q_heads):
    """Ranges of positions that a tile of 128 rows is cut into: two workgroups a compute unit, 16 at most."""
    tiles = B.rows * (q_heads // B.heads) // 128 + len(B.new)
    return min(16, max(1, 2 * _units() // (tiles * B.heads)))


def _cache(B, std_code=120):
    """Finite codes everywhere that a position is, scales around 2^(std_code - 127)."""
    kv, scale = B.ref.kv, B.ref.scale
    kv[(kv & 0x7F) == 0x7F] = 0x29
    scale[:] = B.rng.integers(std_code - 2, std_code + 1, scale.shape)
    return kv, scale


def _send(B):
    B.kv.copy_(torch.from_numpy(B.ref.kv))
    B.scale.copy_(torch.from_numpy(B.ref.scale))


def _want(B, q, scale, causal=True, window=0):
    rows, heads, dim = q.shape
    g = heads // B.heads
    q = q.cuda().double()
    out, mag = (torch.zeros(rows, heads, dim, dtype=torch.float64, device="cuda") for _ in range(2))
    lse, reach = (torch.zeros(rows, heads, dtype=torch.float64, device="cuda") for _ in range(2))
    table = TABLE.cuda()
    for b, n in enumerate(B.new):
        lo, end = int(B.starts[b]), int(B.lens[b])
        if not n:
            continue
        t, p = torch.arange(end, device="cuda"), torch.arange(end - n, end, device="cuda")[:, None]
        page = torch.from_numpy(B.table[b]).cuda().long()[t // B.page]
        there = (page >= 0) & (page < B.kv.shape[1])
        at = torch.where(there, page, 0)
        see = there & (t < end) & ((t <= p) if causal else torch.ones_like(t <= p))
        if window:
            see = see & (t > p - window)
        code = B.scale[:, at, :, t % B.page // 16].double()  # [end][2][heads], indexed dimensions first
        unit = torch.where(code == 255, float("nan"), torch.exp2(code - 127))
        vals = table[B.kv[:, at, :, t % B.page].long()] * unit[..., None]
        for h in range(heads):
            k, v = vals[:, 0, h // g].contiguous(), vals[:, 1, h // g].contiguous()
            qh = q[lo:lo + n, h].contiguous()
            s = torch.where(see, qh @ k.t().contiguous() * scale, float("-inf"))
            m = s.amax(1, keepdim=True)
            e = torch.exp(s - torch.where(torch.isinf(m), 0, m))
            total = e.sum(1, keepdim=True)
            odd = ~torch.isfinite(v)
            bad = (see.double() @ odd.double()) > 0  # NaN only where the row sees it
            w = e / torch.where(total > 0, total, 1)
            out[lo:lo + n, h] = torch.where(bad, float("nan"), w @ torch.where(odd, 0, v))
            mag[lo:lo + n, h] = w @ torch.where(odd, 0, v).abs()
            lse[lo:lo + n, h] = (m + torch.log(total))[:, 0]
            reach[lo:lo + n, h] = torch.where(see, qh.abs() @ k.abs().t().contiguous(), 0).amax(1) * scale
    return tuple(x.cpu().numpy() for x in (out, lse, mag, reach))


def _compare(mx, B, q_heads, std=1.0, scale=None, causal=True, window=0, max_new=0, q=None):
    q = bf16(B.rng, B.rows, q_heads, B.dim, std=std) if q is None else q
    scale = B.dim ** -0.5 if scale is None else scale
    out, lse = mx.mx_kv_attention(q.cuda(), *B.args, scale=scale, causal=causal, window=window, max_new=max_new, want_lse=True)
    want = _want(B, q, scale, causal, window)
    check_attention(out, lse, want, B.dim, int(B.lens.max()))
    return out


def _nan_places(B):
    """NaN codes and scales: in the middle, in the last rows' own positions, where no window of 150 from the end reaches."""
    kv, scale = B.ref.kv, B.ref.scale

    def cell(b, p):
        return B.table[b, p // B.page], p % B.page

    for b, end in enumerate(B.lens):
        for w, p, h in ((0, end // 2, 0), (1, end // 3, 0), (1, end - 1, B.heads - 1), (0, end - 2, B.heads - 1)):
            pg, slot = cell(b, int(p))
            kv[w, pg, h, slot, 7] = 0xFF
        pg, slot = cell(b, int(end) // 4)
        scale[1, pg, B.heads - 1, slot // 16] = 255


PROMPTS = [
    # new rows, positions before them, kv heads, q heads, dim, page, ranges
    ([260, 210, 300, 250], [150, 333, 201, 400], 8, 32, 128, 64, (1, 1)),
    ([760, 500], [0, 299], 4, 28, 64, 16, (1, 1)),
    ([600, 520], [500, 460], 4, 16, 128, 32, (2, 4)),
    ([700, 1, 600], [450, 900, 777], 3, 15, 64, 128, (2, 4)),
]


@pytest.mark.parametrize("new,ctx,kv_heads,q_heads,dim,page,ranges", PROMPTS)
def test_prompts_of_many_steps(gpu_lib, new, ctx, kv_heads, q_heads, dim, page, ranges):
    """At least six steps of 64 positions for a workgroup: the buffers' turns, the running maximum past them, the rows
    stored without a join and joined from a few ranges."""
    B = Batch(sum(new), new, ctx, kv_heads, dim, page, filled=False)
    _cache(B)
    _send(B)
    n = _ranges(B, q_heads)
    assert ranges[0] <= n <= ranges[1] and max(c + a for c, a in zip(ctx, new)) // 64 // n >= 3 * 2 ** (n == 1)
    _compare(gpu_lib, B, q_heads, std=0.3)
    _compare(gpu_lib, B, q_heads, std=2.0, max_new=max(new))
    _compare(gpu_lib, B, q_heads, causal=False)
    _compare(gpu_lib, B, q_heads, window=390)
    _compare(gpu_lib, B, q_heads, window=129)
    # keys that grow step by step: the maximum is raised again and again, over accumulators that hold something
    for b, end in enumerate(B.lens):
        for p in range(0, int(end), 16):
            B.ref.scale[0, B.table[b, p // page], :, p % page // 16] = 124 - min((int(end) - 1 - p) // 64, 18)
    _send(B)
    _compare(gpu_lib, B, q_heads, std=1.5)
    _cache(B)
    _nan_places(B)
    _send(B)
    for kw in (dict(), dict(window=150), dict(causal=False)):
        got = _compare(gpu_lib, B, q_heads, **kw)
        assert torch.isnan(got).any() and not torch.isnan(got).all()


STEPS = [
    # new rows a sequence, sequences, kv heads, q heads, dim, page
    (1, 12, 8, 32, 128, 64),
    (1, 24, 4, 12, 64, 16),
    (4, 13, 8, 48, 128, 32),
    (6, 20, 4, 28, 64, 16),
]


@pytest.mark.parametrize("new,batch,kv_heads,q_heads,dim,page", STEPS)
def test_pieces_that_cross_items(gpu_lib, new, batch, kv_heads, q_heads, dim, page):
    """Sequences of uneven lengths on a line of many more chunks than pieces: pieces of several chunks, some of which end
    one item and start the next; two tiles of rows at once where a head has over 16 (dim 128 and 64)."""
    rng = np.random.default_rng(batch)
    ctx = [int(c) for c in rng.integers(200, 5600, batch)]
    counts = [new if b % 5 else 1 for b in range(batch)]
    B = Batch(new + batch, counts, ctx, kv_heads, dim, page, filled=False)
    _cache(B)
    _send(B)
    rows = new * (q_heads // kv_heads)
    tiles = [-(-n * (q_heads // kv_heads) // (16 if rows <= 16 else 32)) for n in counts]
    chunks = [-(-int(e) // 128) for e in B.lens]
    line = kv_heads * sum(t * c for t, c in zip(tiles, chunks))
    piece = -(-line // (2 * _units()))
    assert piece >= 3 and any(c % piece for c in chunks) and max(chunks) > 3 * piece
    _compare(gpu_lib, B, q_heads, std=0.3, max_new=new)
    _compare(gpu_lib, B, q_heads, std=2.0, max_new=new)
    _compare(gpu_lib, B, q_heads, causal=False, max_new=new)
    _compare(gpu_lib, B, q_heads, window=1500, max_new=new)
    if new == 1:
        _compare(gpu_lib, B, q_heads)  # (not told the most rows: two tiles at once, the prompts' kernel beside it)
    _nan_places(B)
    _send(B)
    for kw in (dict(), dict(window=150), dict(window=1500)):
        got = _compare(gpu_lib, B, q_heads, max_new=new, **kw)
        assert torch.isnan(got).any() and not torch.isnan(got).all()


def test_prompts_beside_single_tokens(gpu_lib):
    """Both kernels in one call, each with several steps or chunks a workgroup."""
    counts = [400, 1, 1, 2, 350, 0, 1, 333]
    B = Batch(77, counts, [300, 5000, 700, 3100, 0, 50, 2222, 411], 4, 128, 64, filled=False)
    _cache(B)
    _send(B)
    assert _ranges(B, 16) <= 4
    for kw in (dict(), dict(window=600), dict(max_new=400)):
        _compare(gpu_lib, B, 16, **kw)
