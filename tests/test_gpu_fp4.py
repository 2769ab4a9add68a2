"""MXFP4 quantization, its inverse and the MXFP4 products against the 64-bit
reference (tests/fp4_ref.py): codes and scales byte for byte.

Products: E2M1 products are multiples of 1/4 up to 36, so a 32-block's sum is
exact in the matrix cores; adding the K/32 block sums (in any order, split
over waves or not) rounds or truncates to FP32 once each, and the split adds a
few more: |C - exact| <= (K/32 + 16) * 2^-23 * sum |a||b|, plus 2^-8 of the
value for BF16.
"""
import numpy as np
import pytest
import torch

import fp4_ref as ref
import mxsynth
import oracle

pytestmark = pytest.mark.gpu

dev = "cuda"


def _np(t):
    return t.cpu().numpy()


def _scales(s_swz, rows, kb):
    return oracle.scale_unswizzle(_np(s_swz).reshape(-1)[:((rows + 31) // 32) * (kb // 8) * 256], rows, kb)


def _check_rowwise(mx, bits):
    rows, cols = bits.shape
    q, s = mx.mx_quantize_rowwise_fp4(mxsynth.from_bits(bits).to(dev))
    codes, scales = ref.quantize(bits)
    assert np.array_equal(_scales(s, rows, cols // 32), scales)
    got = ref.unpack(_np(q))
    assert np.array_equal(got, codes), np.argwhere(got != codes)[:5]
    for dt in (torch.bfloat16, torch.float32):
        y = mx.mx_dequantize_fp4(q, s, out_dtype=dt).double().cpu().numpy()
        want = ref.values(codes, scales)
        assert np.array_equal(y, want, equal_nan=True)
        assert np.array_equal(np.signbit(y[~np.isnan(y)]), np.signbit(want[~np.isnan(want)]))
    return q, s


def test_every_mantissa_exponent_and_sign(gpu_lib):
    """Blocks of every largest exponent whose elements run over every mantissa
    at exponents from the largest down to where everything rounds to zero."""
    rng = np.random.default_rng(0)
    rows = []
    for e in list(range(0, 255)):
        vals = np.array([(max(e - d, 0) << 7) | m for d in range(6) for m in range(128)], np.uint16)
        vals = rng.permutation(vals)
        top = np.uint16((e << 7) | rng.integers(0, 128))
        blocks = np.concatenate([vals, vals[:192 - (len(vals) % 31) % 31]])[:31 * 24].reshape(24, 31)
        blk = np.concatenate([np.full((24, 1), top, np.uint16), blocks], 1)
        blk ^= (rng.integers(0, 2, blk.shape) << 15).astype(np.uint16)
        rows.append(blk.reshape(3, 256))
    _check_rowwise(gpu_lib, np.concatenate(rows))


def test_special_blocks(gpu_lib):
    b = mxsynth.bits(mxsynth.normal_bf16((40, 512), 1.0, seed=3)).copy()
    b[0, :32] = 0
    b[1, :32] = 0x8000
    b[2, 5] = 0x7FC0       # NaN
    b[3, 40] = 0x7F80      # Inf
    b[4, 70] = 0xFF80
    b[5, :] = 0x0001       # smallest subnormal
    b[6, :] = 0x7F7F       # largest finite
    b[7, 33] = 0xFFFF
    _check_rowwise(gpu_lib, b)


def test_dequantize_every_code_and_scale(gpu_lib):
    mx = gpu_lib
    q = np.tile(np.arange(16, dtype=np.uint8), (256, 16))          # [256][256] codes
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, 1)
    y = mx.mx_dequantize_fp4(torch.from_numpy(ref.pack(q)).to(dev), torch.from_numpy(oracle.scale_swizzle(s)).to(dev),
                             out_dtype=torch.float32).cpu().numpy()
    with np.errstate(over="ignore"):
        want = ref.values(q, s).astype(np.float32)
    assert np.array_equal(y, want, equal_nan=True)


@pytest.mark.parametrize("rows,cols", [(1, 256), (31, 512), (33, 768), (257, 2048), (1000, 256)])
def test_quantize_rowwise_shapes(gpu_lib, rows, cols):
    x = mxsynth.normal_bf16((rows, cols), 0.3, seed=rows, outlier_frac=0.01, outlier_mul=100.0)
    _check_rowwise(gpu_lib, mxsynth.bits(x))


def test_quantize_rowwise_views_and_larger_buffer(gpu_lib):
    mx = gpu_lib
    x = mxsynth.normal_bf16((70, 1024), 1.0, seed=9).to(dev)
    q = torch.full((70, 300), 0xA5, dtype=torch.uint8, device=dev)[:, 16:16 + 256]
    s = torch.full((3 * 7 * 256,), 0xA5, dtype=torch.uint8, device=dev)
    with pytest.raises(mx.MxError):
        mx.mx_quantize_rowwise_fp4(x[:, 8:520], q=q, s_swz=s, s_tiles=7)      # rows of 300 bytes
    big = torch.full((70, 304), 0xA5, dtype=torch.uint8, device=dev)
    q = big[:, 16:16 + 256]
    mx.mx_quantize_rowwise_fp4(x[:, 8:520], q=q, s_swz=s, s_tiles=7)
    q2, s2 = mx.mx_quantize_rowwise_fp4(x[:, 8:520].contiguous())
    assert torch.equal(q, q2) and (big[:, :16] == 0xA5).all() and (big[:, 272:] == 0xA5).all()
    t, t2 = s.view(3, 7, 256), s2.view(3, 2, 256)
    assert (t[:, 2:] == 0xA5).all()
    assert torch.equal(t[:2, :2], t2[:2])
    last = _np(t[2, :2].reshape(2, 2, 32, 4)[:, :, :6])
    assert np.array_equal(last, _np(t2[2].reshape(2, 2, 32, 4)[:, :, :6]))
    assert (t[2, :2].reshape(2, 2, 32, 4)[:, :, 6:] == 0xA5).all()            # padding rows are not written


@pytest.mark.parametrize("count,rows,cols", [(1, 256, 32), (1, 512, 96), (3, 256, 2048), (2, 1536, 160), (128, 256, 64)])
def test_quantize_colwise(gpu_lib, count, rows, cols):
    mx = gpu_lib
    x = mxsynth.normal_bf16((count, rows, cols), 0.3, seed=cols, outlier_frac=0.01, outlier_mul=100.0)
    b = mxsynth.bits(x).copy()
    b[0, 3, 1] = 0x7F80
    b[0, :32, 2] = 0x8000
    x = mxsynth.from_bits(b).to(dev)
    qt, st = mx.mx_quantize_colwise_fp4(x if count > 1 else x[0])
    per = mx.mx_scale_swizzled_bytes(cols, rows // 32)
    for i in range(count):
        codes, scales = ref.quantize(np.ascontiguousarray(b[i].T))
        got = _np(qt[i] if count > 1 else qt)
        assert np.array_equal(ref.unpack(got), codes)
        assert np.array_equal(_np(st[i * per:(i + 1) * per]), oracle.scale_swizzle(scales))


def test_quantize_colwise_strided(gpu_lib):
    mx = gpu_lib
    x = mxsynth.normal_bf16((512, 200), 1.0, seed=4).to(dev)
    big = torch.full((160, 320), 0xA5, dtype=torch.uint8, device=dev)
    qt, st = mx.mx_quantize_colwise_fp4(x[:, 8:168], qt=big[:, 32:288])
    q2, s2 = mx.mx_quantize_colwise_fp4(x[:, 8:168].contiguous())
    assert torch.equal(qt, q2) and torch.equal(st, s2)
    assert (big[:, :32] == 0xA5).all() and (big[:, 288:] == 0xA5).all()


def test_dispatch_and_swiglu(gpu_lib):
    mx = gpu_lib
    rng = np.random.default_rng(12)
    for T, H, E, k in ((1, 256, 4, 2), (77, 512, 16, 4), (500, 2048, 128, 8)):
        ids = np.stack([rng.choice(E, size=k, replace=False) for _ in range(T)]).astype(np.int32)
        ids[rng.random(ids.shape) < 0.05] = -1
        x = mxsynth.normal_bf16((T, H), 1.0, seed=T).to(dev)
        idd = torch.from_numpy(ids).to(dev)
        q0 = torch.full((T * k, H // 2), 0xA5, dtype=torch.uint8, device=dev)
        off, src, slot, q, s = mx.mx_moe_dispatch_fp4(x, idd, E, q=q0)
        off8, src8, slot8, _, _ = mx.mx_moe_dispatch(x, idd, E)
        n = int(off[-1])
        assert torch.equal(off, off8) and torch.equal(slot, slot8) and torch.equal(src[:n], src8[:n])
        codes, scales = ref.quantize(mxsynth.bits(x)[_np(src[:n])])
        assert np.array_equal(ref.unpack(_np(q[:n])), codes)
        assert np.array_equal(_scales(s, T * k, H // 32)[:n], scales)
        assert (q[n:] == 0xA5).all()
    for rows, F in ((1, 256), (37, 768), (300, 1024)):
        gu = mxsynth.normal_bf16((rows, 2 * F), 1.0, seed=F).to(dev)
        q, s, h = mx.mx_swiglu_quantize_fp4(gu, want_h=True)
        _, _, h8 = mx.mx_swiglu_quantize(gu, want_h=True)
        assert torch.equal(h.view(torch.int16), h8.view(torch.int16))
        q2, s2 = mx.mx_quantize_rowwise_fp4(h)
        assert torch.equal(q, q2)
        assert np.array_equal(_scales(s, rows, F // 32), _scales(s2, rows, F // 32))
        q3, s3, none = mx.mx_swiglu_quantize_fp4(gu)
        assert none is None and torch.equal(q3, q)


# ---------------------------------------------------------------------------
# products


def _operand(rng, rows, K, wide=False):
    """Codes of every value; scales over 2^+-6 (wide: blocks up to 2^40 apart)."""
    codes = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    s = rng.integers(107 if wide else 121, 147 if wide else 134, (rows, K // 32)).astype(np.uint8)
    return codes, s


def _dev(codes, s):
    return torch.from_numpy(ref.pack(codes)).to(dev), torch.from_numpy(oracle.scale_swizzle(s)).to(dev)


def _assert_close(C, A, B, K, what):
    want, size = A @ B.T, np.abs(A) @ np.abs(B).T
    got = C.double().cpu().numpy()
    tol = (K / 32 + 16) * 2.0 ** -23 * size + (2.0 ** -8 * np.abs(want) if C.dtype == torch.bfloat16 else 0)
    bad = np.abs(got - want) > tol + 1e-37
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[:4].tolist()}"


SHAPES = [(1, 16, 256), (1, 1, 256), (1, 513, 1024), (3, 48, 256), (16, 64, 512), (17, 100, 768), (48, 33, 2048),
          (64, 256, 1536), (65, 256, 1536), (100, 300, 256), (128, 128, 512), (255, 257, 1280), (256, 256, 256),
          (257, 512, 768), (333, 1000, 2560), (600, 264, 4096)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm(gpu_lib, M, N, K):
    mx = gpu_lib
    rng = np.random.default_rng(M * N + K)
    a, sa = _operand(rng, M, K)
    b, sb = _operand(rng, N, K)
    A, B = ref.values(a, sa), ref.values(b, sb)
    qa, da = _dev(a, sa)
    qb, db = _dev(b, sb)
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.full((M + 1, N), 7.0, dtype=dt, device=dev)
        C = mx.mx_gemm_fp4(qa, da, qb, db, c=buf[:M])
        _assert_close(C, A, B, K, f"{M}x{N}x{K} {dt}")
        assert (buf[M] == 7).all()
        assert torch.equal(C, mx.mx_gemm_fp4(qa, da, qb, db, out_dtype=dt))


@pytest.mark.parametrize("M,N,K", [(5, 96, 1024), (300, 520, 2048)])
def test_gemm_wide_scales_and_nan(gpu_lib, M, N, K):
    mx = gpu_lib
    rng = np.random.default_rng(M)
    a, sa = _operand(rng, M, K, wide=True)
    b, sb = _operand(rng, N, K, wide=True)
    C = mx.mx_gemm_fp4(*_dev(a, sa), *_dev(b, sb), out_dtype=torch.float32)
    _assert_close(C, ref.values(a, sa), ref.values(b, sb), K, "wide")
    sa[2, 3] = 0xFF       # one NaN block: its row of C, nothing else
    sb[7, 1] = 0xFF
    D = mx.mx_gemm_fp4(*_dev(a, sa), *_dev(b, sb), out_dtype=torch.float32)
    nan = torch.zeros(M, N, dtype=torch.bool, device=dev)
    nan[2] = True
    nan[:, 7] = True
    assert torch.equal(torch.isnan(D), nan)
    assert torch.equal(D[~nan], C[~nan])


@pytest.mark.parametrize("M", [7, 290])
def test_gemm_strides(gpu_lib, M):
    mx = gpu_lib
    rng = np.random.default_rng(M)
    N, K = 272, 1024
    a, sa = _operand(rng, M, K)
    b, sb = _operand(rng, N, K)
    qa, da = _dev(a, sa)
    qb, db = _dev(b, sb)
    wa = torch.full((M, K // 2 + 48), 0x77, dtype=torch.uint8, device=dev)
    wb = torch.full((N, K // 2 + 16), 0x77, dtype=torch.uint8, device=dev)
    wa[:, 16:16 + K // 2] = qa
    wb[:, :K // 2] = qb
    ref_ = mx.mx_gemm_fp4(qa, da, qb, db)
    for pad, off in ((0, 0), (8, 8), (5, 3), (1, 0)):
        buf = torch.full((M, N + off + pad), 9.0, dtype=torch.bfloat16, device=dev)
        mx.mx_gemm_fp4(wa[:, 16:16 + K // 2], da, wb[:, :K // 2], db, c=buf[:, off:off + N])
        got = buf[:, off:off + N]
        # a C of other alignment may be summed in another split
        assert (got.float() - ref_.float()).abs().max() <= 2.0 ** -7 * ref_.float().abs().max()
        _assert_close(got, ref.values(a, sa), ref.values(b, sb), K, f"pad {pad}")
        assert (buf[:, :off] == 9).all() and (buf[:, off + N:] == 9).all()


GROUPED = [(3, [0, 1, 5], 40, 256), (4, [1, 0, 0, 1], 1536, 2048), (5, [3, 70, 0, 16, 130], 257, 512),
           (8, [300, 0, 17, 256, 1, 255, 257, 64], 320, 768), (2, [0, 0], 64, 256), (1, [33], 48, 1024),
           (128, None, 96, 256)]


@pytest.mark.parametrize("G,rows,N,K", GROUPED)
def test_grouped_gemm(gpu_lib, G, rows, N, K):
    mx = gpu_lib
    rng = np.random.default_rng(G * N + K)
    if rows is None:
        rows = rng.integers(0, 9, G).tolist()
    tail = 5                                   # rows of A behind the last expert's
    off = np.concatenate([[0], np.cumsum(rows)]).astype(np.int64)
    M = int(off[-1]) + tail
    a, sa = _operand(rng, M, K)
    bs = [_operand(rng, N, K) for _ in range(G)]
    qa, da = _dev(a, sa)
    qb = torch.from_numpy(np.stack([ref.pack(b) for b, _ in bs])).to(dev)
    db = torch.from_numpy(np.concatenate([oracle.scale_swizzle(s) for _, s in bs])).to(dev)
    A = ref.values(a, sa)
    for dt in (torch.bfloat16, torch.float32):
        C = torch.full((M, N), 7.0, dtype=dt, device=dev)
        mx.mx_grouped_gemm_fp4(torch.from_numpy(off).to(dev), qa, da, qb, db, c=C)
        for g in range(G):
            lo, hi = off[g], off[g + 1]
            if hi > lo:
                _assert_close(C[lo:hi], A[lo:hi], ref.values(*bs[g]), K, f"expert {g}")
        assert (C[int(off[-1]):] == 7).all()


def test_grouped_offsets_out_of_order_stay_in_bounds(gpu_lib):
    """Offsets that break their properties give unspecified values inside C only."""
    mx = gpu_lib
    rng = np.random.default_rng(2)
    G, N, K, M = 4, 96, 256, 50
    a, sa = _operand(rng, M, K)
    bs = [_operand(rng, N, K) for _ in range(G)]
    qb = torch.from_numpy(np.stack([ref.pack(b) for b, _ in bs])).to(dev)
    db = torch.from_numpy(np.concatenate([oracle.scale_swizzle(s) for _, s in bs])).to(dev)
    buf = torch.full((M + 20, N), 7.0, device=dev)
    for off in ([0, 40, 10, 60, 50], [-5, 10, 1000, 20, 50], [0, 0, 0, 0, 10 ** 12]):
        mx.mx_grouped_gemm_fp4(torch.tensor(off, dtype=torch.int64, device=dev), *_dev(a, sa), qb, db, c=buf[:M])
        torch.cuda.synchronize()
        assert (buf[M:] == 7).all()
