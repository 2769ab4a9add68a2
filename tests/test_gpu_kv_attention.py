"""Attention over the paged 8-bit cache against the loops of tests/kv_ref.py;
tolerances: tests/kv_util.py (attention_bounds)."""
import numpy as np
import pytest
import torch

from kv_util import BF, Batch, attention_bounds, bf16, check_attention

pytestmark = pytest.mark.gpu


def _run(mx, B, q_heads, std=1.0, scale=None, causal=True, window=0, max_new=0, q=None, want=None):
    q = bf16(B.rng, B.rows, q_heads, B.dim, std=std) if q is None else q
    out = torch.full((B.rows, q_heads, B.dim), 7.0, dtype=BF, device="cuda")
    lse = torch.full((B.rows, q_heads), 7.0, device="cuda")
    got = mx.mx_kv_attention(q.cuda(), *B.args, scale=scale, causal=causal, window=window, max_new=max_new, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    torch.cuda.synchronize()
    n = int(B.starts[-1])
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()  # rows behind the last sequence
    if want is None:
        want = B.ref.attention(q.double().numpy()[:n], B.starts, B.lens, B.dim ** -0.5 if scale is None else scale, causal, window)
    check_attention(out[:n], lse[:n], want, B.dim, int(min(max(B.lens.max(), 1), B.table.shape[1] * B.page)))
    return out[:n], lse[:n], want


STEPS = [
    # new rows, positions before them, kv heads, q heads, dim, page, layout
    ([1], [0], 1, 1, 64, 16, "hnd"),
    ([1], [0], 2, 8, 128, 64, "hnd"),
    ([1, 1, 1], [14, 15, 16], 2, 8, 128, 16, "hnd"),
    ([1, 0, 1, 1], [127, 5, 128, 129], 1, 7, 64, 32, "nhd"),
    ([1, 1], [700, 33], 2, 10, 128, 64, "alternate"),
    ([1], [1300], 1, 16, 64, 128, "padded"),
    ([1], [300], 1, 20, 128, 16, "hnd"),
    ([1], [200], 1, 40, 64, 64, "hnd"),
    ([1], [100], 1, 64, 64, 256, "hnd"),
    ([3, 5, 1], [40, 0, 260], 2, 6, 64, 16, "hnd"),
    ([4, 2], [500, 17], 2, 16, 128, 32, "nhd"),
    ([7], [90], 3, 9, 128, 1024, "hnd"),
]


# a table of up to 1024 positions keeps a sequence's work together, a larger one lets it be cut over the chip
ROOM = [0, 1500]


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("new,ctx,kv_heads,q_heads,dim,page,layout", STEPS)
def test_few_rows(gpu_lib, new, ctx, kv_heads, q_heads, dim, page, layout, room):
    B = Batch(sum(ctx) + dim + q_heads, new, ctx, kv_heads, dim, page, layout, behind=3, room=room)
    _run(gpu_lib, B, q_heads, max_new=max(new))
    _run(gpu_lib, B, q_heads, std=4.0, max_new=max(new) + 2)
    _run(gpu_lib, B, q_heads, causal=False, scale=0.3)
    _run(gpu_lib, B, q_heads, window=20, max_new=max(new))


PROMPTS = [
    ([65], [0], 1, 1, 64, 16, "hnd"),
    ([40], [0], 2, 8, 128, 64, "hnd"),
    ([129, 3], [0, 20], 1, 2, 128, 32, "nhd"),
    ([70, 1, 0, 33], [15, 200, 9, 64], 2, 6, 64, 16, "hnd"),
    ([200], [130], 1, 1, 128, 128, "alternate"),
    ([17, 90], [63, 1], 1, 5, 64, 64, "padded"),
    ([9], [50], 1, 33, 128, 16, "hnd"),
]


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("new,ctx,kv_heads,q_heads,dim,page,layout", PROMPTS)
def test_many_rows(gpu_lib, new, ctx, kv_heads, q_heads, dim, page, layout, room):
    B = Batch(sum(ctx) + dim + q_heads, new, ctx, kv_heads, dim, page, layout, behind=2, room=room)
    _run(gpu_lib, B, q_heads, max_new=max(new))
    _run(gpu_lib, B, q_heads, std=4.0)
    _run(gpu_lib, B, q_heads, causal=False, scale=0.2)
    _run(gpu_lib, B, q_heads, window=37)


def test_long_rows_split_over_the_chip(gpu_lib):
    """One row a head over many pieces; a torch reference in 64 bits on the device's values."""
    for dim, page, ctx, heads, kv_heads in ((128, 64, 9000, 8, 2), (64, 16, 20011, 3, 1)):
        B = Batch(dim, [1], [0], kv_heads, dim, page, filled=False)
        pages = -(-(ctx + 1) // page)
        g = torch.Generator(device="cuda").manual_seed(3)
        kv = torch.randint(0, 255, (2, pages, kv_heads, page, dim), generator=g, device="cuda").to(torch.uint8)
        kv[(kv & 127) == 127] = 0x30
        scale = torch.randint(118, 121, (2, pages, kv_heads, page // 16), generator=g, device="cuda").to(torch.uint8)
        table = torch.randperm(pages, generator=g, device="cuda").int()[None]
        lens = torch.tensor([ctx + 1], dtype=torch.int32, device="cuda")
        starts = torch.tensor([0, 1], device="cuda")
        q = bf16(B.rng, 1, heads, dim, std=0.05)
        out, lse = gpu_lib.mx_kv_attention(q.cuda(), kv, scale, table, lens, starts, max_new=1, want_lse=True)
        vals = kv.view(torch.float8_e4m3fn).double() * torch.exp2(scale.double() - 127).repeat_interleave(16, 3)[..., None]
        vals = vals[:, table[0].long()].transpose(2, 3).reshape(2, -1, kv_heads, dim)[:, :ctx + 1].cpu().numpy()
        qn = q.double().numpy()
        want, wl, mag, reach = np.zeros(q.shape), np.zeros((1, heads)), np.zeros(q.shape), np.zeros((1, heads))
        for h in range(heads):
            k, v = vals[0, :, h * kv_heads // heads], vals[1, :, h * kv_heads // heads]
            s = k @ qn[0, h] * dim ** -0.5
            e = np.exp(s - s.max())
            want[0, h], mag[0, h], wl[0, h] = e @ v / e.sum(), e @ np.abs(v) / e.sum(), s.max() + np.log(e.sum())
            reach[0, h] = (np.abs(k) @ np.abs(qn[0, h])).max() * dim ** -0.5
        check_attention(out, lse, (want, wl, mag, reach), dim, ctx + 1)


def test_rows_that_see_nothing(gpu_lib):
    """Sequences without positions, rows at positions below 0, pages that are not there."""
    for rows, room in ((2, 0), (90, 0), (2, 1500), (90, 1500)):
        B = Batch(31, [rows, rows, 3, rows], [0, 30, 0, 20], 2, 64, 16, behind=1, room=room)
        B.lens[0] = 0            # nothing in the cache
        B.lens[2] = 1            # two rows at positions below 0
        B.table[3, :] = -1       # no page at all
        B.table[1, 0] = 10 ** 6  # one page missing
        for kw in (dict(), dict(causal=False), dict(window=5), dict(max_new=rows)):
            out, lse, want = _run(gpu_lib, B, 4, **kw)
            assert (out[:rows] == 0).all() and torch.isneginf(lse[:rows]).all()
    B.lens[:] = -5
    out, lse, _ = _run(gpu_lib, B, 4)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("rows", [1, 5, 70])
def test_nan_and_infinities_in_masked_places(gpu_lib, rows, room):
    """A position's NaN reaches the rows that see it, and no other: behind the last position, behind
    a causal row, before a window, in a missing page."""
    B = Batch(32 + rows, [rows, rows], [33, 0], 2, 64, 16, behind=1, room=room)
    kv, sc = B.ref.kv, B.ref.scale

    def cell(b, p):
        return B.table[b, p // 16], p % 16

    n0, n1 = 33 + rows, rows
    for w in range(2):
        pg, slot = cell(0, n0 - 1)
        kv[w, pg, 1, slot, 3] = 0x7F      # the last position of sequence 0: its own row sees it
        pg, slot = cell(0, 2)
        kv[w, pg, 0, slot, 9] = 0xFF      # an early one, outside a window of 20
    if rows > 4:
        pg, slot = cell(1, n1 - 3)
        kv[1, pg, 0, slot, :] = 0x7F
        pg, slot = cell(1, n1 - 2)
        kv[0, pg, 1, slot, 5] = 0x7F
        sc[1, cell(1, 0)[0], 1, 0] = 254  # scales past BF16's range: infinite values in the block
    sc[0, cell(0, 16)[0], 0, 0] = 255     # a block of NaN keys
    B.kv.copy_(torch.from_numpy(kv))
    B.scale.copy_(torch.from_numpy(sc))
    q = bf16(B.rng, B.rows, 4, 64)
    for kw in (dict(), dict(window=20), dict(window=3), dict(max_new=rows)):
        out = gpu_lib.mx_kv_attention(q.cuda(), *B.args, want_lse=True, **kw)
        n = int(B.starts[-1])
        with np.errstate(invalid="ignore", over="ignore"):
            want = B.ref.attention(q.double().numpy()[:n], B.starts, B.lens, 0.125, True, kw.get("window", 0))
        # a block's scale of 2^127: codes below 2 in magnitude are values from 2^118 to 2^128, finite in BF16, larger
        # ones infinite; a sum of weights up to 2^8 with the former may overflow before it is divided
        big = np.abs(want[0]) > 1e30
        got = out[0][:n].double().cpu().numpy()
        with np.errstate(invalid="ignore", over="ignore"):
            near = np.abs(got - want[0]) <= attention_bounds(*want, 64, 200)[0]
        assert (near | ~np.isfinite(got))[big].all()
        got[big], want[0][big], want[2][big] = 0.0, 0.0, 0.0
        check_attention(torch.from_numpy(got), out[1][:n], want, 64, 200)


def test_scale_zero_and_peaked_rows(gpu_lib):
    B = Batch(33, [1, 40], [50, 9], 1, 64, 32)
    for scale in (0.0, 1e-30, 3.0):
        _run(gpu_lib, B, 2, scale=scale)
    # scores far apart, growing along the positions: the running maximum moves at every step
    ref = B.ref
    for p in range(51):
        pg, slot = B.table[0, p // 32], p % 32
        ref.kv[0, pg, 0, slot] = 0x38
        ref.scale[0, pg, 0, slot // 16] = 120 + p // 16
    B.kv.copy_(torch.from_numpy(ref.kv))
    B.scale.copy_(torch.from_numpy(ref.scale))
    _run(gpu_lib, B, 2, scale=20.0, q=torch.ones(B.rows, 2, 64).to(BF))


def test_strided_queries_and_outputs(gpu_lib):
    for new in ([1, 2], [50, 3]):
        B = Batch(34, new, [20, 5], 2, 128, 64)
        qkv = bf16(B.rng, B.rows, 8, 128).cuda()
        for q in (qkv[:, 2:6], qkv.transpose(0, 1).contiguous().transpose(0, 1)[:, :4]):
            want = gpu_lib.mx_kv_attention(q.contiguous(), *B.args)
            wide = torch.full((B.rows, 9, 136), 3.0, dtype=BF, device="cuda")
            got = gpu_lib.mx_kv_attention(q, *B.args, out=wide[:, 3:7, :128])
            assert torch.equal(got, want)
            wide[:, 3:7, :128] = 3.0
            assert (wide == 3.0).all()


def test_same_call_same_bytes(gpu_lib):
    for new, ctx, room in (([1] * 9, [700, 3, 64, 1500, 0, 99, 130, 400, 31], 0), ([150, 20], [40, 300], 0),
                           ([150, 3], [40, 300], 1500)):
        B = Batch(35, new, ctx, 2, 128, 32, filled=False, room=room)
        B.scale.fill_(118)
        B.kv[(B.kv & 127) == 127] = 0x11
        q = bf16(B.rng, B.rows, 8, 128).cuda()
        first = gpu_lib.mx_kv_attention(q, *B.args, want_lse=True)
        need = gpu_lib.mx_kv_attention_workspace_bytes(B.rows, len(new), 8, 2, 128)
        for fill in (0, 255):
            ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
            again = gpu_lib.mx_kv_attention(q, *B.args, want_lse=True, workspace=ws)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_without_rounding_only_weights_are_lost(gpu_lib):
    """One visible position: its value comes back exactly, whatever the scores."""
    B = Batch(36, [1, 1], [0, 0], 2, 64, 16)
    out, lse, _ = _run(gpu_lib, B, 4, std=9.0)
    v = B.ref.read(B.starts, B.lens, 2)[1]
    assert np.array_equal(out.double().cpu().numpy(), np.repeat(v, 2, 1))


def test_many_sequences_bad_starts_and_small_max_new(gpu_lib):
    rng = np.random.default_rng(37)
    new = [int(n) for n in rng.integers(0, 3, 600)]
    B = Batch(37, new, [int(n) for n in rng.integers(0, 40, 600)], 1, 64, 16, filled=False, room=1500)
    B.ref.scale[:] = 120
    B.ref.kv[(B.ref.kv & 127) == 127] = 0x21
    B.kv.copy_(torch.from_numpy(B.ref.kv))
    B.scale.fill_(120)
    _run(gpu_lib, B, 3, max_new=2)
    _run(gpu_lib, B, 3)
    kv, scale, table, lens, starts = B.args
    q = bf16(rng, B.rows, 3, 64).cuda()
    bad = starts.flip(0).contiguous()
    bad[5], bad[400] = -9, 10 ** 13
    for kw in (dict(), dict(max_new=1), dict(max_new=100)):
        gpu_lib.mx_kv_attention(q, kv, scale, table, lens, bad, **kw)
        gpu_lib.mx_kv_attention(q, kv, scale, table, lens * 1000000, starts, **kw)
    torch.cuda.synchronize()


def test_lengths_past_the_table(gpu_lib):
    """kv_lens far beyond what the table holds: positions from there on are not stored, windows there are empty."""
    B = Batch(39, [2, 70, 1], [30, 0, 5], 1, 64, 16, room=1100)
    cap = B.table.shape[1] * 16
    for lens in ([2 ** 31 - 1, cap + 1, 2 ** 31 - 3], [cap, cap + 40, cap + 2]):
        B.lens = np.array(lens, np.int32)
        for kw in (dict(window=1), dict(window=33), dict(window=2 ** 40), dict(causal=False), dict(max_new=70)):
            _run(gpu_lib, B, 2, **kw)


def test_binding_refusals(gpu_lib):
    B = Batch(38, [2, 3], [0, 9], 2, 64, 16)
    q = bf16(B.rng, 5, 4, 64).cuda()
    kv, scale, table, lens, starts = B.args
    good = dict(q=q, kv=kv, kv_scale=scale, page_table=table, kv_lens=lens, seq_starts=starts)
    f32 = dict(dtype=torch.float32, device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(q=q[..., :32]), dict(out=q.float()), dict(out=q[:4]),
                dict(lse=torch.empty(5, 3, **f32)), dict(lse=torch.empty(5, 4, dtype=BF, device="cuda")),
                dict(workspace=torch.empty(1 << 24, dtype=torch.uint8)), dict(kv_lens=lens.cpu())):
        with pytest.raises(ValueError):
            gpu_lib.mx_kv_attention(**dict(good, **bad))
    for bad in (dict(q=bf16(B.rng, 5, 3, 64).cuda()), dict(scale=-1.0), dict(window=3, causal=False), dict(window=-1),
                dict(max_new=-1), dict(out=q), dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(gpu_lib.MxError):
            gpu_lib.mx_kv_attention(**dict(good, **bad))
    assert gpu_lib.mx_kv_attention(q[:0], kv, scale, table, lens, starts * 0).shape == (0, 4, 64)


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("rows", [12, 70])
def test_nan_value_scales(gpu_lib, rows, room):
    """A block of values whose scale is NaN, beside blocks that are none: rows that see only those get numbers."""
    clean = 0
    for dim, at in ((64, 16), (128, 16), (64, 32), (128, 32), (64, 48)):
        if at >= 33 + rows:
            continue
        B = Batch(40 + rows + at, [rows, 3], [33, 20], 2, dim, 16, room=room)
        B.ref.scale[1, B.table[0, at // 16], 0, 0] = 255
        B.scale.copy_(torch.from_numpy(B.ref.scale))
        for kw in (dict(), dict(window=10), dict(window=3), dict(max_new=rows)):
            out, _, _ = _run(gpu_lib, B, 4, **kw)
            clean += int(torch.isfinite(out[:rows, :2].float()).all(-1).all(-1).sum())
    assert clean  # (some row sees nothing of the block)


def test_windows_that_reach_far(gpu_lib):
    """Windows from 2^30 on, rows as far: positions are numbers below 2^31, whatever the table holds."""
    B = Batch(41, [2, 70], [30, 0], 1, 64, 16, room=1100)
    cap = B.table.shape[1] * 16
    for lens in ([2 ** 31 - 1, 2 ** 31 - 1], [2 ** 30 + 40, 2 ** 30 + 71]):
        B.lens = np.array(lens, np.int32)
        for window in (2 ** 30 - 1, 2 ** 30, 2 ** 30 + 20, 2 ** 31 - 40, 2 ** 31 - 2, 2 ** 31 - 1, 2 ** 31, 2 ** 62):
            _run(gpu_lib, B, 2, window=window)
            _run(gpu_lib, B, 2, window=window, max_new=70)
    assert cap < 2 ** 30


def test_values_at_the_ends_of_the_scales(gpu_lib):
    """One visible position: the value comes back as mx_kv_read's BF16, subnormal and infinite ones too."""
    codes = [0, 1, 2, 3, 5, 8, 246, 247, 248, 254]
    n = len(codes)
    for rows, kv_heads in ((1, 4), (70, 4)):
        B = Batch(42, [1] * n, [0] * n, kv_heads, 64, 16, filled=False)
        flat = np.arange(kv_heads * 64) % 256
        flat[(flat & 127) == 127] = 0x31
        B.ref.scale[0] = 120
        B.ref.kv[0] = 0x38
        for b, c in enumerate(codes):
            B.ref.kv[1, B.table[b, 0], :, 0] = flat.reshape(kv_heads, 64)
            B.ref.scale[1, B.table[b, 0]] = c
        B.kv.copy_(torch.from_numpy(B.ref.kv))
        B.scale.copy_(torch.from_numpy(B.ref.scale))
        _, v = gpu_lib.mx_kv_read(*B.args, n)
        q = bf16(B.rng, n, kv_heads * rows, 64).cuda()
        out = gpu_lib.mx_kv_attention(q, *B.args)
        assert torch.isinf(v).any() and (v[v != 0].abs().min() < 2.0 ** -130)
        assert torch.equal(out, v.repeat_interleave(rows, 1)), rows


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("dim,group", [(64, 1), (64, 16), (128, 7)])
def test_single_tokens_keep_their_weights(gpu_lib, dim, group, room):
    """Up to 16 rows a head: a weight reaches the product with the values as two BF16 numbers, off by 2^-8 of 2^-8 of
    itself, so the outputs are as near as their own rounding and the FP32 sums let them (attention_bounds without the 2^-8 of
    the weights).  With a NaN outside a window too, where positions go one by one."""
    kv_heads = 2
    ctx = [int(c) for c in np.random.default_rng(43).integers(14, 60, 8)]
    B = Batch(43 + dim + group, [1] * 8, ctx, kv_heads, dim, 16, room=room)
    q = bf16(B.rng, 8, kv_heads * group, dim, std=0.1)
    for window in (0, 12):
        if window:
            for b in range(8):
                B.ref.kv[1, B.table[b, 0], :, 1] = 0x7F
            B.kv.copy_(torch.from_numpy(B.ref.kv))
        out = gpu_lib.mx_kv_attention(q.cuda(), *B.args, window=window, max_new=1).double().cpu().numpy()
        want, _, mag, reach = ref = B.ref.attention(q.double().numpy(), B.starts, B.lens, dim ** -0.5, True, window)
        assert np.isfinite(want).all()
        bound = attention_bounds(*ref, dim, int(B.lens.max()))[0] - 2.0 ** -8 * mag + 2.0 ** -16 * mag
        err = np.abs(out - want)
        assert (err <= bound).all(), ((err > bound).sum(), (err / bound).max())
