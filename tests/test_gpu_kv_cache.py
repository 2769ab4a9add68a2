"""Appending to the paged 8-bit cache and reading it back, against the loops of
tests/kv_ref.py: codes and scales are whole numbers and must be equal (the
rotation is formed in 64 bits on both sides, and E4M3 is its only rounding)."""
import numpy as np
import pytest
import torch

import kv_ref as ref
from kv_util import BF, Batch, bf16

pytestmark = pytest.mark.gpu


def _append(mx, B, k, v, freqs=None, rows=None, **kw):
    fd = None if freqs is None else torch.from_numpy(freqs).cuda()
    mx.mx_kv_append(k, v, *B.args, freqs=fd, **kw)
    B.ref.append(k.double().cpu().numpy(), v.double().cpu().numpy(), B.starts, B.lens, freqs, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(B.scale_np(), B.ref.scale), "scales differ"
    got, want = B.kv_np(), B.ref.kv
    assert np.array_equal(got, want), f"{(got != want).sum()} codes differ, first {np.argwhere(got != want)[:3]}"


def _freqs(rot, base=1e4):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


CASES = [
    # new rows, positions before them, heads, dim, page, layout
    ([1], [0], 1, 64, 16, "hnd"),
    ([1], [15], 1, 128, 16, "hnd"),
    ([1, 1, 1], [16, 31, 100], 2, 128, 64, "nhd"),
    ([40, 3, 17], [0, 5, 31], 3, 64, 32, "hnd"),
    ([5, 0, 1, 0, 33], [7, 20, 0, 0, 15], 2, 128, 16, "alternate"),
    ([129], [3], 1, 64, 1024, "padded"),
    ([16, 16], [16, 8], 8, 128, 128, "hnd"),
    ([2] * 21, list(range(21)), 5, 64, 32, "nhd"),
]


@pytest.mark.parametrize("style", [None, "half", "interleaved"])
@pytest.mark.parametrize("new,ctx,heads,dim,page,layout", CASES)
def test_append_and_read(gpu_lib, new, ctx, heads, dim, page, layout, style):
    B = Batch(sum(new) + dim + page, new, ctx, heads, dim, page, layout, behind=2)
    k, v = bf16(B.rng, B.rows, heads, dim, std=3.0), bf16(B.rng, B.rows, heads, dim)
    k[:, 0, 5] *= 40
    if style is None:
        _append(gpu_lib, B, k.cuda(), v.cuda())
    else:
        _append(gpu_lib, B, k.cuda(), v.cuda(), _freqs(dim if style == "half" else 32, 1e6), style=style, amplitude=1.25)
    for dtype in (BF, torch.float32):
        gk, gv = (torch.full((B.rows, heads, dim), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        assert gpu_lib.mx_kv_read(*B.args, B.rows, k=gk, v=gv)[0] is gk
        want = B.ref.read(B.starts, B.lens, B.rows)
        n = B.rows - 2
        for got, w in ((gk, want[0]), (gv, want[1])):
            assert np.array_equal(got[:n].double().cpu().numpy(), w[:n])  # exact in both types
            assert (got[n:] == 7.0).all()  # rows behind the last sequence


def test_whole_sequences_come_back(gpu_lib):
    B = Batch(5, [0, 0, 0], [37, 0, 90], 2, 64, 32)
    B.starts = np.concatenate([[0], np.cumsum(B.lens)]).astype(np.int64)
    rows = int(B.lens.sum())
    k, v = gpu_lib.mx_kv_read(*B.args, rows, out_dtype=torch.float32)
    assert np.array_equal(np.stack([k.double().cpu().numpy(), v.double().cpu().numpy()]), B.ref.read(B.starts, B.lens, rows))


def test_a_block_grows_token_by_token(gpu_lib):
    """One token at a time, growing: the scale grows, older codes are rounded anew; a new block starts anew."""
    B = Batch(8, [1], [0], 2, 64, 16, spare=3)
    B.table = np.array([[1, 3, 0]], np.int32)
    B.ref.table = B.table
    rng = np.random.default_rng(1)
    seen = set()
    for p in range(40):
        B.lens[:] = p + 1
        k, v = bf16(rng, 1, 2, 64, std=2.0 ** (p % 16 - 3)).cuda(), bf16(rng, 1, 2, 64, std=2.0 ** (5 - p % 16)).cuda()
        _append(gpu_lib, B, k, v, _freqs(64))
        seen.add(int(B.ref.scale[0, B.table[0, p // 16], 0, 0]))
    assert len(seen) > 5
    # back to a position inside a block: its scale stays, older codes too
    B.lens[:] = 20
    _append(gpu_lib, B, bf16(rng, 1, 2, 64).cuda(), bf16(rng, 1, 2, 64).cuda())


def test_special_values(gpu_lib):
    B = Batch(9, [20, 3], [5, 0], 2, 64, 32)
    k, v = bf16(B.rng, 23, 2, 64), bf16(B.rng, 23, 2, 64)
    k[2, 0, 7], k[4, 1, :], k[20, 1, 9] = float("nan"), float("inf"), float("-inf")
    v[3, 0, 1], v[22], v[21, 1, :] = float("inf"), 0.0, -0.0
    v[6, 1, :3] = torch.tensor([3.3895e38, -3.3895e38, 1e-38])
    v[:, 0, 60] = 1e-40
    k[21:23, 0] = 0.0  # a block of zeros but for one row
    k[20, 0] = 2.0 ** -133
    _append(gpu_lib, B, k.cuda(), v.cuda())
    _append(gpu_lib, B, k.cuda(), v.cuda(), _freqs(64), amplitude=2.0)
    gk, _ = gpu_lib.mx_kv_read(*B.args, 23)
    assert torch.isnan(gk[4, 1]).any()


def test_ties_and_the_top_of_the_range(gpu_lib):
    """Midpoints go to the even code; 448 and just above it choose the scale."""
    B = Batch(10, [16, 16, 16], [0, 0, 0], 1, 64, 16)
    x = torch.zeros(48, 1, 64)
    mid = torch.from_numpy((ref.E4M3[:126] + ref.E4M3[1:127]) / 2).float()
    x[:2, 0, :] = mid[:126].reshape(2, 63)[:, list(range(63)) + [0]]
    x[2, 0, 0] = 448.0
    x[16:18] = x[:2]
    x[18, 0, 0] = 450.0
    x[32, 0, 0] = -452.0
    k = x.to(BF)
    _append(gpu_lib, B, k.cuda(), (-k).cuda())
    assert B.ref.scale[0, B.table[0, 0], 0, 0] == 127 and B.ref.scale[0, B.table[1, 0], 0, 0] == 128


def test_rotated_keys_beside_midpoints(gpu_lib):
    """Rotated by a multiple of a quarter turn to within 2^-50, keys at the midpoints of two codes land just beside them: a
    rounding to FP32 on the way would make ties of them."""
    B = Batch(21, [32], [0], 1, 64, 32)
    mid = torch.from_numpy((ref.E4M3[8:126] + ref.E4M3[9:127]) / 2).float()
    k = torch.ones(32, 1, 64) * 2.0 ** -9
    k[:, 0, :32] = mid[torch.randint(0, 118, (32, 32), generator=torch.Generator().manual_seed(2))]
    k[:, 0, 0] = 448.0
    f = np.full(32, 2 * np.pi * 2.0 ** -31) * np.arange(32)  # angles of 2^-29 and less
    _append(gpu_lib, B, k.to(BF).cuda(), k.to(BF).cuda(), f)


def test_strided_rows(gpu_lib):
    """Keys and values as parts of one projection's output, and heads outside the rows."""
    new, ctx, heads, dim = [3, 20], [30, 9], 2, 128
    for kind in (0, 1):
        B = Batch(12, new, ctx, heads, dim, 64)
        qkv = bf16(B.rng, 23, 6, dim).cuda()
        k, v = (qkv[:, 2:4], qkv[:, 4:]) if kind == 0 else (qkv.transpose(0, 1).contiguous().transpose(0, 1)[:, i:i + 2] for i in (0, 3))
        _append(gpu_lib, B, k, v, _freqs(128))


def test_pages_that_are_not_there(gpu_lib):
    """Page numbers out of range, positions below 0 or past the table: nothing is stored, zeros come back."""
    B = Batch(13, [50, 40, 10], [40, 0, 0], 2, 64, 16)
    B.table[0, 3] = -1
    B.table[0, 4] = 10 ** 6
    B.table[1, 1] = B.kv.shape[1]
    B.lens[1] = 30       # 40 rows, the first ten at positions below 0
    B.lens[2] = 16 * B.table.shape[1] + 4  # the last four past the table
    B.table[2, :] = -1
    B.table[2, -1] = B.table[2, -1] if False else [p for p in range(B.kv.shape[1]) if p not in B.table[:2]][0]
    k, v = bf16(B.rng, 100, 2, 64).cuda(), bf16(B.rng, 100, 2, 64).cuda()
    _append(gpu_lib, B, k, v, _freqs(64))
    gk, gv = gpu_lib.mx_kv_read(*B.args, 100)
    want = B.ref.read(B.starts, B.lens, 100)
    assert np.array_equal(gk.double().cpu().numpy(), want[0]) and np.array_equal(gv.double().cpu().numpy(), want[1])
    assert (want[:, 50:60] == 0).all() and (want[:, -4:] == 0).all()


def test_nan_scales_read_as_nan(gpu_lib):
    B = Batch(14, [0], [20], 1, 64, 16)
    B.starts[1] = 20
    for scale in (B.ref.scale, ):
        scale[1, B.table[0, 0], 0, 0] = 255
    B.scale.copy_(torch.from_numpy(B.ref.scale))
    k, v = gpu_lib.mx_kv_read(*B.args, 20)
    assert torch.isnan(v[:16]).all() and torch.isfinite(v[16:]).all() and torch.isfinite(k).all()


def test_many_sequences_and_bad_starts(gpu_lib):
    """More sequences than a workgroup's threads, empty ones among them; starts that break
    their properties stay in bounds."""
    rng = np.random.default_rng(15)
    new = [int(n) for n in rng.integers(0, 3, 700)]
    B = Batch(16, new, [int(n) for n in rng.integers(0, 20, 700)], 1, 64, 16, filled=False)
    k, v = bf16(rng, B.rows, 1, 64).cuda(), bf16(rng, B.rows, 1, 64).cuda()
    # (blocks that hold any bytes before the call: their scales too)
    B.ref.scale[:] = 120
    B.scale.fill_(120)
    _append(gpu_lib, B, k, v)
    kv, scale, table, lens, starts = B.args
    bad = starts.flip(0).contiguous()
    bad[3], bad[500] = -7, 10 ** 12
    gpu_lib.mx_kv_append(k, v, kv, scale, table, lens, bad)
    gpu_lib.mx_kv_read(kv, scale, table, lens, bad, B.rows)
    torch.cuda.synchronize()


def test_debug_checks_the_starts(gpu_lib, monkeypatch):
    B = Batch(17, [3, 4], [0, 0], 1, 64, 16)
    k = bf16(B.rng, 7, 1, 64).cuda()
    kv, scale, table, lens, starts = B.args
    monkeypatch.setenv("MX_DEBUG", "1")
    gpu_lib.mx_kv_append(k, k, kv, scale, table, lens, starts)
    for bad in ([0, 5, 4], [1, 3, 7], [0, 3, 9]):
        b = torch.tensor(bad).cuda()
        for call in (lambda: gpu_lib.mx_kv_append(k, k, kv, scale, table, lens, b), lambda: gpu_lib.mx_kv_read(kv, scale, table, lens, b, 7),
                     lambda: gpu_lib.mx_kv_attention(k, kv, scale, table, lens, b)):
            with pytest.raises(gpu_lib.MxError, match="seq_starts") as e:
                call()
            assert e.value.status == gpu_lib.MX_ERR_INVALID_ARG


def test_binding_refusals(gpu_lib):
    B = Batch(18, [2, 3], [0, 9], 2, 64, 16)
    k = bf16(B.rng, 5, 2, 64).cuda()
    kv, scale, table, lens, starts = B.args
    good = dict(k=k, v=k.clone(), kv=kv, kv_scale=scale, page_table=table, kv_lens=lens, seq_starts=starts)
    for bad in (dict(k=k.float()), dict(v=k[:4]), dict(v=k[:, :1]), dict(kv=kv[:1]), dict(kv=kv.to(torch.int8)), dict(kv=kv[0]),
                dict(kv_scale=scale[:, :-1]), dict(page_table=table.long()), dict(page_table=table[0]), dict(kv_lens=lens[:1]),
                dict(kv_lens=lens.long()), dict(seq_starts=starts[:2]), dict(seq_starts=starts.int()), dict(kv_scale=scale.cpu()),
                dict(style="none"), dict(freqs=torch.ones(32).cuda()), dict(kv=kv.transpose(3, 4))):
        with pytest.raises(ValueError):
            gpu_lib.mx_kv_append(**dict(good, **bad))
    for bad in (dict(freqs=torch.ones(40, dtype=torch.float64).cuda()), dict(freqs=torch.ones(4, dtype=torch.float64).cuda())):
        with pytest.raises(gpu_lib.MxError):
            gpu_lib.mx_kv_append(**dict(good, **bad))
    with pytest.raises(ValueError):
        gpu_lib.mx_kv_read(kv, scale, table, lens, starts, 5, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        gpu_lib.mx_kv_read(kv, scale, table, lens, starts, 5, k=torch.empty(5, 2, 64).cuda(), v=torch.empty(5, 2, 64).cuda().bfloat16())
    empty = Batch(19, [0, 0], [3, 4], 2, 64, 16)
    gpu_lib.mx_kv_append(k[:0], k[:0], *empty.args)
    assert gpu_lib.mx_kv_read(*empty.args, 0)[0].shape == (0, 2, 64)


def test_debug_checks_the_most_rows(gpu_lib, monkeypatch):
    """MX_DEBUG finds a sequence with more rows than max_new says."""
    B = Batch(22, [3, 4, 0], [0, 5, 9], 1, 64, 16)
    q = bf16(B.rng, 7, 1, 64).cuda()
    monkeypatch.setenv("MX_DEBUG", "1")
    for most in (0, 4, 5, 1 << 40):
        gpu_lib.mx_kv_attention(q, *B.args, max_new=most)
    for most, at in ((3, 1), (2, 0), (1, 0)):
        with pytest.raises(gpu_lib.MxError, match=rf"max_new.*seq_starts\[{at}\]") as e:
            gpu_lib.mx_kv_attention(q, *B.args, max_new=most)
        assert e.value.status == gpu_lib.MX_ERR_INVALID_ARG


def test_reading_at_the_ends_of_the_scales(gpu_lib):
    """Every finite code at the smallest and the largest scales: FP32 holds the value, or is infinite beyond its range;
    BF16 rounds to nearest where its last bit (2^-133) does not reach."""
    codes = [0, 1, 2, 3, 4, 7, 8, 120, 127, 200, 246, 247, 248, 250, 254]
    B = Batch(23, [0], [16 * len(codes)], 1, 64, 16, filled=False)
    B.starts[1] = B.lens[0]
    flat = np.arange(16 * 64) % 256
    flat[(flat & 127) == 127] = 0x31
    for i, c in enumerate(codes):
        B.ref.kv[:, B.table[0, i], 0] = flat.reshape(16, 64)
        B.ref.scale[:, B.table[0, i], 0, 0] = c
    B.kv.copy_(torch.from_numpy(B.ref.kv))
    B.scale.copy_(torch.from_numpy(B.ref.scale))
    rows = int(B.lens[0])
    want = B.ref.read(B.starts, B.lens, rows)
    with np.errstate(over="ignore"):
        f32 = want.astype(np.float32)  # exact, or infinite
    assert (np.isinf(f32) | (f32 == want)).all() and np.isinf(f32).any()
    # to nearest even by hand: the step of a BF16 value is 2^(exponent - 7), 2^-133 at least; beyond FP32's range infinite
    with np.errstate(divide="ignore"):
        step = 2.0 ** np.maximum(np.floor(np.log2(np.abs(want))) - 7, -133)
    near = np.where(np.isinf(f32), f32, np.rint(want / step) * step)
    assert (near != want)[:, :48].any() and (near == want)[:, 48:][np.isfinite(f32[:, 48:])].all()
    for dtype, w in ((torch.float32, f32), (BF, near)):
        k, v = gpu_lib.mx_kv_read(*B.args, rows, out_dtype=dtype)
        for got, x in ((k, w[0]), (v, w[1])):
            assert np.array_equal(got.double().cpu().numpy(), x.astype(np.float64)), dtype


def test_the_largest_values_come_back_infinite(gpu_lib):
    """A finite value that rounds to 2^128 is beyond FP32 when it is read: from 248 * 2^120 on, whose tie goes to the even
    code."""
    B = Batch(24, [4], [0], 1, 64, 16)
    x = torch.zeros(4, 1, 64)
    for i, m in enumerate((240, 247, 248, 255)):
        x[i] = m * 2.0 ** 120
        x[i, :, 1::2] *= -1
    k = x.to(BF)
    assert torch.equal(k.float(), x)
    _append(gpu_lib, B, k.cuda(), (-k).cuda())
    gk, gv = gpu_lib.mx_kv_read(*B.args, 4)
    want = x.double()
    want[1] = want[0]
    want[2:] *= float("inf")
    assert torch.equal(gk.double().cpu(), want) and torch.equal(gv.double().cpu(), -want)
