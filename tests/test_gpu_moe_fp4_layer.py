"""The routing and MXFP4 operators together, as a MoE layer's forward and
backward and a sampler's step use them; captured and replayed; on several
streams; and products large enough for every way that the library cuts them.

Each stage is checked against its 64-bit definition on the stage's own inputs
(what the stage before wrote on the GPU), so no tolerance compounds.  Product
tolerance: (K/32 + 16) * 2^-23 * sum |a||b|, plus 2^-8 of the value for BF16
(tests/test_gpu_fp4.py derives it).
"""
import numpy as np
import pytest
import torch

import fp4_ref as ref
import mxsynth
import oracle

pytestmark = pytest.mark.gpu

dev = "cuda"
VALUE = [0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6]


def _decode(q, s_swz):
    """FP64 values on the GPU, by table and by the layout's definition."""
    rows, half = q.shape
    k = 2 * half
    table = torch.tensor(VALUE, dtype=torch.float64, device=dev)
    v = table[torch.stack([q & 15, q >> 4], -1).reshape(rows, k).long()]
    blk = torch.arange(k // 32, device=dev)
    row = torch.arange(rows, device=dev)[:, None]
    at = ((row // 32) * (k // 256) + blk // 8) * 256 + (32 * (blk % 2) + row % 32) * 4 + blk % 8 // 2
    return v * torch.exp2(s_swz[at].double() - 127).repeat_interleave(32, dim=1)


def _close(C, A, B, what):
    K = A.shape[1]
    want, size = A @ B.t(), A.abs() @ B.abs().t()
    tol = (K / 32 + 16) * 2.0 ** -23 * size + (2.0 ** -8 * want.abs() if C.dtype == torch.bfloat16 else 0)
    bad = (C.double() - want).abs() > tol + 1e-37
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[:4].tolist()}"


def _random_operand(g, rows, K):
    q = torch.randint(0, 256, (rows, K // 2), generator=g, device=dev, dtype=torch.uint8)
    s = torch.randint(121, 134, ((rows + 31) // 32 * (K // 256) * 256,), generator=g, device=dev, dtype=torch.uint8)
    return q, s


# ---------------------------------------------------------------------------
# every way a product is cut


@pytest.mark.parametrize("M,N,K,split", [
    (1, 4096, 12288, False), (30, 4096, 4096, False), (60, 4096, 4096, False),    # few rows: 16, 32, 64 a pass
    (64, 24576, 512, False), (333, 6144, 1024, False), (1000, 4096, 512, False),  # 128 x 128 tiles
    (200, 4096, 12288, True), (90, 1024, 8192, True),                             # and split along K
    (2048, 4096, 2048, False), (2000, 4104, 2304, False),                         # 256 x 128
    (2048, 8192, 2048, False), (4096, 4096, 8192, False),                         # 256 x 256
    (4608, 4096, 12288, True),
    (2044, 94, 14592, True), (90, 1001, 8192, True), (131, 130, 5120, True)])     # split, columns left over
def test_products_cut_every_way(gpu_lib, M, N, K, split):
    mx = gpu_lib
    g = torch.Generator(device=dev)
    g.manual_seed(M + N + K)
    a, sa = _random_operand(g, M, K)
    b, sb = _random_operand(g, N, K)
    assert (mx.mx_gemm_fp4_workspace_bytes(M, N, K) > 0) == split
    A, B = _decode(a, sa), _decode(b, sb)
    for dt in (torch.bfloat16, torch.float32):
        C = mx.mx_gemm_fp4(a, sa, b, sb, out_dtype=dt)
        _close(C, A, B, f"{M}x{N}x{K} {dt}")
        assert torch.equal(C, mx.mx_gemm_fp4(a, sa, b, sb, out_dtype=dt))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(200, 4096, 12288), (77, 1001, 8192)])
def test_split_products_into_unaligned_rows(gpu_lib, M, N, K, dt):
    """C of any alignment and leading dimension; what is around it stays."""
    mx = gpu_lib
    g = torch.Generator(device=dev)
    g.manual_seed(M)
    a, sa = _random_operand(g, M, K)
    b, sb = _random_operand(g, N, K)
    assert mx.mx_gemm_fp4_workspace_bytes(M, N, K, dt) > 0
    want = mx.mx_gemm_fp4(a, sa, b, sb, out_dtype=dt)
    for left, right in ((0, 1), (1, 2), (3, 4), (8, 8)):
        buf = torch.full((M + 1, left + N + right), 7.0, dtype=dt, device=dev)
        mx.mx_gemm_fp4(a, sa, b, sb, c=buf[:M, left:left + N])
        assert torch.equal(buf[:M, left:left + N], want)
        buf[:M, left:left + N] = 7.0
        assert (buf == 7.0).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(333, 1000, 1024), (2000, 4103, 2304), (4097, 4095, 4096), (700, 50, 768), (1500, 513, 256)])
def test_products_into_unaligned_rows(gpu_lib, M, N, K, dt):
    """The same of every tile size, several tiles a workgroup, unsplit or with a split rest."""
    mx = gpu_lib
    g = torch.Generator(device=dev)
    g.manual_seed(M)
    a, sa = _random_operand(g, M, K)
    b, sb = _random_operand(g, N, K)
    A, B = _decode(a, sa), _decode(b, sb)
    want = None
    for left, right in ((1, 2), (0, 0), (3, 5), (2, 1)):
        buf = torch.full((M + 1, left + N + right), 7.0, dtype=dt, device=dev)
        mx.mx_gemm_fp4(a, sa, b, sb, c=buf[:M, left:left + N])
        if want is None:
            want = buf[:M, left:left + N].clone()
            _close(want, A, B, f"{M}x{N}x{K}")
        assert torch.equal(buf[:M, left:left + N], want)
        buf[:M, left:left + N] = 7.0
        assert (buf == 7.0).all()


@pytest.mark.parametrize("rows,N,K", [
    ([150] + [1] * 50 + [0] * 13, 96, 512),           # few rows: an expert of three chunks
    ([0, 0, 1, 0], 200, 256), ([16] * 4, 48, 768),
    ([300, 0, 17, 129, 1, 128, 127, 90], 1000, 512),  # 128 x 128 tiles
    ([700, 300, 0, 513], 520, 1024),                  # 256 x 256
    ([384, 385, 383, 641, 256, 513, 1025, 320], 776, 768),   # and tails of every kind: whole, half or less
    ([128, 900, 1, 1152, 127, 0, 129, 500], 256, 256), ([2000, 64, 65, 63], 512, 1280),
    ([900, 3, 2500, 1100, 129, 4000, 31, 0], 4097, 2048), ([40, 300, 1, 77], 1001, 1024),   # and rows of odd length
    ([0] * 1023 + [5], 64, 256)])
def test_grouped_products_cut_every_way(gpu_lib, rows, N, K):
    mx = gpu_lib
    G = len(rows)
    g = torch.Generator(device=dev)
    g.manual_seed(G + N)
    off = np.concatenate([[0], np.cumsum(rows)])
    M = int(off[-1])
    a, sa = _random_operand(g, M, K)
    n32 = (N + 31) // 32 * 32
    b = torch.randint(0, 256, (G, N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    sb = torch.randint(121, 134, (G, n32 * (K // 32)), generator=g, device=dev, dtype=torch.uint8)
    A = _decode(a, sa)
    for dt in (torch.bfloat16, torch.float32):
        C = mx.mx_grouped_gemm_fp4(torch.from_numpy(off).to(dev), a, sa, b, sb, out_dtype=dt)
        for e in range(G):
            if rows[e]:
                _close(C[off[e]:off[e + 1]], A[off[e]:off[e + 1]], _decode(b[e], sb[e]), f"expert {e}")


def test_large_buffers(gpu_lib):
    """C, x and q beyond 2^32 bytes: the rows at both ends."""
    mx = gpu_lib
    g = torch.Generator(device=dev)
    g.manual_seed(3)
    M, N, K = 150_001, 16384, 256
    a, sa = _random_operand(g, M, K)
    b, sb = _random_operand(g, N, K)
    C = mx.mx_gemm_fp4(a, sa, b, sb)
    assert C.numel() * 2 > 1 << 32
    B = _decode(b, sb)
    for lo in (0, M - 300):
        _close(C[lo:lo + 300], _decode(a, sa)[lo:lo + 300], B, f"rows from {lo}")
    q, s = mx.mx_quantize_rowwise_fp4(C)
    for lo in (0, M // 32 * 32 - 256):
        q2, s2 = mx.mx_quantize_rowwise_fp4(C[lo:lo + 256])
        assert torch.equal(q[lo:lo + 256], q2)
        assert torch.equal(s.view(-1, N // 256 * 256)[lo // 32:lo // 32 + 8], s2.view(8, -1))
    x = mx.mx_dequantize_fp4(q, s)
    assert torch.equal(x[-5:], mx.mx_dequantize_fp4(q[M // 32 * 32:], s[M // 32 * N:])[-5:])


def test_more_rows_than_a_launch_takes(gpu_lib):
    """More than 2^31 units of 16 bytes: several launches a call.  The last rows
    and those around the cuts equal the same rows in small calls."""
    mx = gpu_lib
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB of free device memory")
    R, C = (1 << 22) + 40, 4096
    g = torch.Generator(device=dev)
    g.manual_seed(6)
    base = torch.randn(R // 8, 64, generator=g, device=dev).bfloat16()
    gu = torch.empty(R, 2 * C, dtype=torch.bfloat16, device=dev)
    gu.view(R // 8, -1, 64).copy_(base[:, None])             # rows 8i .. 8i + 7 repeat 64 values
    gu[-3:].neg_()
    tile = lambda s, r, cols: s.view(-1, cols)[r // 32:(r + 32) // 32]  # noqa: E731  (a 32-row tile has cols scale bytes)
    at = [0, (1 << 22) - 32, 1 << 22]                        # the cut is at row 2^22 (2^21 for FP32 values)
    q, s, _ = mx.mx_swiglu_quantize_fp4(gu)
    for r in at:
        q2, s2, _ = mx.mx_swiglu_quantize_fp4(gu[r:r + 32])
        assert torch.equal(q[r:r + 32], q2) and torch.equal(tile(s, r, C), s2.view(1, -1))
    q2, _, _ = mx.mx_swiglu_quantize_fp4(gu[-8:])
    assert torch.equal(q[-8:], q2)
    x = gu[:, C:]
    q, s = mx.mx_quantize_rowwise_fp4(x, q=q, s_swz=s)
    for r in at:
        q2, s2 = mx.mx_quantize_rowwise_fp4(x[r:r + 32])
        assert torch.equal(q[r:r + 32], q2) and torch.equal(tile(s, r, C), s2.view(1, -1))
    q2, s2 = mx.mx_quantize_rowwise_fp4(x[-8:])
    assert torch.equal(q[-8:], q2)
    y = mx.mx_dequantize_fp4(q, s)
    for r in at:
        assert torch.equal(y[r:r + 32], mx.mx_dequantize_fp4(q[r:r + 32], tile(s, r, C).reshape(-1)))
    assert torch.equal(y[-8:], mx.mx_dequantize_fp4(q2, s2))
    del y
    half = R // 2 + 36                                       # FP32 values: half the rows are a cut
    y = mx.mx_dequantize_fp4(q[:half], s, out_dtype=torch.float32)
    for r in (0, (1 << 21) - 32, 1 << 21):
        assert torch.equal(y[r:r + 32], mx.mx_dequantize_fp4(q[r:r + 32], tile(s, r, C).reshape(-1), out_dtype=torch.float32))
    assert torch.equal(y[-8:].bfloat16(), mx.mx_dequantize_fp4(*mx.mx_quantize_rowwise_fp4(x[half - 8:half])))
    del y
    ids = torch.zeros(R, 1, dtype=torch.int32, device=dev)   # one expert: the rows keep their order
    want_q, want_s = q.clone(), s.clone()
    q.zero_(), s.zero_()
    _, _, slot, q, s = mx.mx_moe_dispatch_fp4(x, ids, 1, q=q, s_swz=s)
    assert torch.equal(slot, torch.arange(R, device=dev, dtype=torch.int32))
    assert torch.equal(q, want_q) and torch.equal(s.view(-1, C)[:-1], want_s.view(-1, C)[:-1])


def test_large_expert_rows_and_stacks(gpu_lib):
    """y, dy, a stack of weights and the grouped product's B beyond 2^32 bytes:
    both ends equal the same rows in a small call."""
    mx = gpu_lib
    g = torch.Generator(device=dev)
    g.manual_seed(8)
    T, k, H = 131_400, 8, 2048
    n = T * k
    y = torch.randint(-32768, 32767, (n, H), generator=g, device=dev, dtype=torch.int16).clamp_(0x3000, 0x4000).view(torch.bfloat16)
    assert y.numel() * 2 > 1 << 32
    d = torch.randn(T, H, generator=g, device=dev).bfloat16()
    w = torch.rand(T, k, generator=g, device=dev)
    slot = torch.arange(n - 1, -1, -1, device=dev, dtype=torch.int32)   # the first token has the last rows
    dy, dw = mx.mx_moe_combine_bwd(d, y, slot, w)
    for lo in (0, T - 4):
        rows = slot[lo * k:(lo + 4) * k].long()
        some = torch.arange(4 * k, device=dev, dtype=torch.int32)
        dy2, dw2 = mx.mx_moe_combine_bwd(d[lo:lo + 4], y[rows], some, w[lo:lo + 4].contiguous())
        assert torch.equal(dy[rows], dy2) and torch.equal(dw[lo:lo + 4], dw2)
    del dy, dw
    G, N, K = 1026, 1024, 2048
    x = y.view(-1)[:G * N * K].view(G, N, K)
    q, s = mx.mx_quantize_colwise_fp4(x)
    per = mx.mx_scale_swizzled_bytes(K, N // 32)
    for e in (0, G - 1):
        q2, s2 = mx.mx_quantize_colwise_fp4(x[e])
        assert torch.equal(q[e], q2) and torch.equal(s[e * per:(e + 1) * per], s2)
    del q, s, x, y
    G, N, K, M = 260, 8192, 4096, 700
    b, sb = _random_operand(g, G * N, K)
    assert b.numel() > 1 << 32
    a, sa = _random_operand(g, M, K)
    for rows in ([1, 3], [300, 400]):          # few rows; tiles
        off = torch.zeros(G + 1, dtype=torch.int64, device=dev)
        off[1:] = rows[0]
        off[G] = sum(rows)
        m = sum(rows)
        C = mx.mx_grouped_gemm_fp4(off, a[:m], sa, b.view(G, N, K // 2), sb)
        A = _decode(a, sa)[:m]
        for e, lo, hi in ((0, 0, rows[0]), (G - 1, rows[0], m)):
            sl = N * K // 32
            _close(C[lo:hi], A[lo:hi], _decode(b[e * N:(e + 1) * N], sb[e * sl:(e + 1) * sl]), f"expert {e} of {rows}")


def test_grouped_debug_check(gpu_lib, monkeypatch):
    mx = gpu_lib
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    a, sa = _random_operand(g, 40, 256)
    b, sb = _random_operand(g, 64, 256)
    b, off = b.view(2, 32, 128), torch.tensor([0, 50, 40], device=dev)
    monkeypatch.setenv("MX_DEBUG", "1")
    with pytest.raises(mx.MxError) as e:
        mx.mx_grouped_gemm_fp4(off, a, sa, b, sb)
    assert e.value.status == mx.MX_ERR_INVALID_ARG and "group_offsets[1]" in str(e.value)
    mx.mx_grouped_gemm_fp4(torch.tensor([0, 15, 40], device=dev), a, sa, b, sb)


# ---------------------------------------------------------------------------
# the layer


def _weights(mx, E, H, F, seed):
    w_gu = mxsynth.normal_bf16((E, 2 * F, H), 0.05, seed=seed).to(dev)
    w_dn = mxsynth.normal_bf16((E, H, F), 0.05, seed=seed + 1).to(dev)
    W = {}
    for name, w in (("gu", w_gu), ("dn", w_dn)):
        q, s = mx.mx_quantize_rowwise_fp4(w.view(-1, w.shape[2]))      # forward operand of every expert
        W[name] = (q.view(E, w.shape[1], -1), s)
        W[name + "_t"] = mx.mx_quantize_colwise_fp4(w)                 # data gradient's
    return W


def _forward(mx, x, logits, W, E, k, o=None, ws=None, stream=None, **route):
    """One MoE layer: (out, everything that the backward keeps)."""
    o = o or {}
    ids, w = mx.mx_moe_route(logits, k, topk_ids=o.get("ids"), weights=o.get("w"), stream=stream, **route)
    off, src, slot, q, s = mx.mx_moe_dispatch_fp4(x, ids, E, offsets=o.get("off"), src=o.get("src"), slot=o.get("slot"),
                                                  q=o.get("q"), s_swz=o.get("s"), workspace=ws, stream=stream)
    gu = mx.mx_grouped_gemm_fp4(off, q, s, *W["gu"], c=o.get("gu"), stream=stream)
    hq, hs, h = mx.mx_swiglu_quantize_fp4(gu, q=o.get("hq"), s_swz=o.get("hs"), h=o.get("h"), want_h=True, stream=stream)
    y = mx.mx_grouped_gemm_fp4(off, hq, hs, *W["dn"], c=o.get("y"), stream=stream)
    out = mx.mx_moe_combine(y, slot, w, out=o.get("out"), stream=stream)
    return out, dict(ids=ids, w=w, off=off, src=src, slot=slot, q=q, s=s, gu=gu, hq=hq, hs=hs, h=h, y=y)


def _backward(mx, d_out, logits, f, W, o=None, **route):
    """(dy, d_weights, d_h, d_logits): what the expert weights' and the layers below need."""
    o = o or {}
    dy, dw = mx.mx_moe_combine_bwd(d_out, f["y"], f["slot"], f["w"], dy=o.get("dy"), d_weights=o.get("dw"))
    dq, ds = mx.mx_quantize_rowwise_fp4(dy, q=o.get("dq"), s_swz=o.get("ds"))
    dh = mx.mx_grouped_gemm_fp4(f["off"], dq, ds, *W["dn_t"], c=o.get("dh"))
    how = {n: route[n] for n in ("score", "renormalize", "scale") if n in route}
    dx = mx.mx_moe_route_bwd(dw, logits, f["ids"], d_logits=o.get("dx"), **how)
    return dict(dy=dy, dw=dw, dq=dq, ds=ds, dh=dh, dx=dx)


@pytest.mark.parametrize("T,E,k,H,F,route", [
    (1, 8, 2, 256, 256, {}),
    (5, 128, 8, 512, 256, dict(score="sigmoid", num_groups=8, topk_groups=4, group_top=2, scale=2.5)),
    (300, 16, 4, 512, 256, dict(renormalize=False)), (2100, 8, 2, 256, 512, {})])
def test_layer_forward_and_backward(gpu_lib, T, E, k, H, F, route):
    mx = gpu_lib
    x = mxsynth.normal_bf16((T, H), 1.0, seed=1, outlier_frac=0.002, outlier_mul=20.0).to(dev)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).to(dev)
    mask = torch.ones(T, dtype=torch.uint8)
    mask[T // 2 + 1:T // 2 + 3] = 0               # padded tokens
    kw = dict(route, mask=mask.to(dev))
    if route.get("score") == "sigmoid":
        kw["bias"] = torch.randn(E, generator=torch.Generator().manual_seed(3)).to(dev) * 0.1
    W = _weights(mx, E, H, F, 5)
    out, f = _forward(mx, x, logits, W, E, k, **kw)
    torch.cuda.synchronize()
    rid, rw = ref.route(logits.cpu().numpy(), k, route.get("score") != "sigmoid",
                        kw["bias"].cpu().numpy() if "bias" in kw else None, route.get("num_groups", 1),
                        route.get("topk_groups", 1), route.get("group_top", 1), route.get("renormalize", True),
                        route.get("scale", 1.0), mask.numpy())
    assert np.array_equal(f["ids"].cpu().numpy(), rid)
    assert np.allclose(f["w"].cpu().numpy(), rw, rtol=2.0 ** -16, atol=0)
    off, src, slot = oracle.moe_dispatch(rid, E)
    n = int(off[-1])
    assert n == int(mask.sum()) * k
    assert np.array_equal(f["off"].cpu().numpy(), off) and np.array_equal(f["slot"].cpu().numpy(), slot)
    codes, scales = ref.quantize(mxsynth.bits(x)[src[:n]])
    assert np.array_equal(ref.unpack(f["q"][:n].cpu().numpy()), codes)
    A, Hd = _decode(f["q"], f["s"])[:n], _decode(f["hq"], f["hs"])[:n]
    tile = mx.mx_scale_swizzled_bytes
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi == lo:
            continue
        _close(f["gu"][lo:hi], A[lo:hi], _decode(W["gu"][0][e], W["gu"][1][e * tile(2 * F, H // 32):]), f"gate_up {e}")
        _close(f["y"][lo:hi], Hd[lo:hi], _decode(W["dn"][0][e], W["dn"][1][e * tile(H, F // 32):]), f"down {e}")
    codes, _ = ref.quantize(mxsynth.bits(f["h"][:n]))
    assert np.array_equal(ref.unpack(f["hq"][:n].cpu().numpy()), codes)
    want = torch.zeros(T, H, dtype=torch.float64, device=dev)
    size = torch.zeros_like(want)
    for j in range(k):
        at = torch.from_numpy(slot.reshape(T, k)[:, j].astype(np.int64)).to(dev)
        live = (at >= 0)[:, None]
        term = torch.where(live, f["w"][:, j:j + 1].double() * f["y"][at.clamp(min=0)].double(), 0.0)
        want, size = want + term, size + term.abs()
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + k * 2.0 ** -23 * size + 1e-38).all()
    assert (out[mask.to(dev) == 0] == 0).all()
    # backward
    d_out = mxsynth.normal_bf16((T, H), 1e-2, seed=9).to(dev)
    b = _backward(mx, d_out, logits, f, W, **route)
    prod = (f["w"].unsqueeze(2) * d_out.float().unsqueeze(1)).bfloat16().view(T * k, H)
    a = torch.from_numpy(slot.astype(np.int64)).to(dev)
    assert torch.equal(b["dy"][a[a >= 0]], prod[a >= 0])
    assert (b["dy"][n:] == 0).all()
    dots = torch.where(a >= 0, (d_out.double().repeat_interleave(k, 0) * f["y"][a.clamp(min=0)].double()).sum(1), 0.0)
    mag = (d_out.double().abs().repeat_interleave(k, 0) * f["y"][a.clamp(min=0)].double().abs()).sum(1)
    assert ((b["dw"].double().view(-1) - dots).abs() <= H * 2.0 ** -24 * mag + 1e-38).all()
    Dq = _decode(b["dq"], b["ds"])
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            _close(b["dh"][lo:hi], Dq[lo:hi], _decode(W["dn_t"][0][e], W["dn_t"][1][e * tile(F, H // 32):]), f"dh {e}")
    dx = ref.route_bwd(logits.cpu().numpy(), rid, b["dw"].cpu().numpy(), route.get("score") != "sigmoid",
                       route.get("renormalize", True), route.get("scale", 1.0))
    top = float(b["dw"].abs().max()) * route.get("scale", 1.0)
    assert np.abs(b["dx"].cpu().numpy() - dx).max() <= 256 * 2.0 ** -24 * top
    assert (b["dx"][mask.to(dev) == 0] == 0).all()


def _buffers(T, E, k, H, F):
    n = T * k
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device=dev)  # noqa: E731
    bf, i32 = torch.bfloat16, torch.int32
    swz = lambda r, c: (r + 31) // 32 * (c // 256) * 256  # noqa: E731
    return dict(ids=z(T, k, dt=i32), w=z(T, k, dt=torch.float32), off=z(E + 1, dt=torch.int64), src=z(n, dt=i32),
                slot=z(n, dt=i32), q=z(n, H // 2), s=z(swz(n, H)), gu=z(n, 2 * F, dt=bf), hq=z(n, F // 2), hs=z(swz(n, F)),
                h=z(n, F, dt=bf), y=z(n, H, dt=bf), out=z(T, H, dt=bf), dy=z(n, H, dt=bf), dw=z(T, k, dt=torch.float32),
                dq=z(n, H // 2), ds=z(swz(n, H)), dh=z(n, F, dt=bf), dx=z(T, E, dt=torch.float32))


@pytest.mark.parametrize("T", [3, 700])
def test_layer_captured_and_replayed(gpu_lib, T):
    """The layer and a dense product with a split, captured; every replay, with
    eager work and clobbered outputs between, gives the eager run's bytes."""
    mx = gpu_lib
    E, k, H, F = 16, 4, 512, 256
    x = mxsynth.normal_bf16((T, H), 1.0, seed=1).to(dev)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).to(dev)
    d_out = mxsynth.normal_bf16((T, H), 1e-2, seed=9).to(dev)
    W = _weights(mx, E, H, F, 5)
    g = torch.Generator(device=dev)
    g.manual_seed(7)
    a, sa = _random_operand(g, 200, 12288)
    b, sb = _random_operand(g, 4096, 12288)
    need = mx.mx_gemm_fp4_workspace_bytes(200, 4096, 12288)
    assert need > 0
    ws = torch.empty(max(need, mx.mx_moe_dispatch_workspace_bytes(T, k, E)), dtype=torch.uint8, device=dev)
    o = _buffers(T, E, k, H, F)
    o["dense"] = torch.zeros(200, 4096, dtype=torch.bfloat16, device=dev)

    def run():
        _, f = _forward(mx, x, logits, W, E, k, o=o, ws=ws)
        _backward(mx, d_out, logits, f, W, o=o)
        mx.mx_gemm_fp4(a, sa, b, sb, c=o["dense"], workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in o.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run()
    skip = {"s", "hs", "ds"}       # (their padding rows are not written: the codes' decoded values cover them)
    for rep in range(3):
        for n, t in o.items():
            t.view(torch.uint8).fill_(0 if n in skip else 0xA5 if n != "dy" else 0)
        ws.fill_(0x5A)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in o.items():
            assert torch.equal(t.view(torch.uint8), want[n].view(torch.uint8)), f"replay {rep}: {n}"
        run()                      # eager work between the replays


def test_streams(gpu_lib):
    """The layer on two streams at once, and by the stream argument from a third."""
    mx = gpu_lib
    T, E, k, H, F = 500, 16, 4, 512, 256
    x = mxsynth.normal_bf16((T, H), 1.0, seed=1).to(dev)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).to(dev)
    W = _weights(mx, E, H, F, 5)
    want, _ = _forward(mx, x, logits, W, E, k)
    g = torch.Generator(device=dev)
    g.manual_seed(7)
    a, sa = _random_operand(g, 200, 12288)
    b, sb = _random_operand(g, 4096, 12288)
    dense = mx.mx_gemm_fp4(a, sa, b, sb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for rep in range(3):
        got = []
        for s in (s1, s2):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(_forward(mx, x, logits, W, E, k)[0])
                got.append(mx.mx_gemm_fp4(a, sa, b, sb))
        third, _ = _forward(mx, x, logits, W, E, k, stream=s1)
        fourth = mx.mx_gemm_fp4(a, sa, b, sb, stream=s2.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want) and torch.equal(got[2], want) and torch.equal(third, want)
        assert torch.equal(got[1], dense) and torch.equal(got[3], dense) and torch.equal(fourth, dense)


def test_binding_refusals(gpu_lib):
    mx = gpu_lib
    x = torch.randn(4, 256, device=dev).bfloat16()
    lg = torch.randn(4, 16, device=dev)
    with pytest.raises(ValueError, match="bias"):
        mx.mx_moe_route(lg, 2, bias=torch.zeros(16))                 # on the host
    with pytest.raises(ValueError, match="bias"):
        mx.mx_moe_route(lg, 2, bias=torch.zeros(15, device=dev))
    with pytest.raises(ValueError, match="score"):
        mx.mx_moe_route(lg, 2, score="relu")
    with pytest.raises(ValueError, match="logits"):
        mx.mx_moe_route(lg.half(), 2)
    with pytest.raises(ValueError, match="logits"):
        mx.mx_moe_route(lg.t(), 2)
    with pytest.raises(mx.MxError, match="topk"):
        mx.mx_moe_route(lg, 17)
    with pytest.raises(ValueError, match="mask"):
        mx.mx_moe_route(lg, 2, mask=torch.ones(4, device=dev))
    ids, w = mx.mx_moe_route(lg, 2)
    with pytest.raises(ValueError, match="d_weights"):
        mx.mx_moe_route_bwd(w[:3], lg, ids)
    with pytest.raises(ValueError, match="d_weights needs y"):
        mx.mx_moe_combine_bwd(x, None, torch.zeros(8, dtype=torch.int32, device=dev), w)
    with pytest.raises(ValueError, match="slot"):
        mx.mx_moe_combine_bwd(x, x.repeat(2, 1), torch.zeros(7, dtype=torch.int32, device=dev), w)
    q, s = mx.mx_quantize_rowwise_fp4(x)
    with pytest.raises(ValueError, match="s_swz"):
        mx.mx_dequantize_fp4(q, s[:100])
    with pytest.raises(mx.MxError) as e:
        mx.mx_quantize_rowwise_fp4(x[:, :128])
    assert e.value.status == mx.MX_ERR_UNSUPPORTED
    with pytest.raises(mx.MxError) as e:
        mx.mx_quantize_colwise_fp4(x[:, :64])
    assert e.value.status == mx.MX_ERR_SHAPE
    with pytest.raises(ValueError, match="b_q"):
        mx.mx_gemm_fp4(q, s, q[:, :64], s)
    with pytest.raises(mx.MxError, match="workspace"):
        g = torch.Generator(device=dev)
        g.manual_seed(1)
        a, sa = _random_operand(g, 200, 12288)
        b, sb = _random_operand(g, 4096, 12288)
        mx.mx_gemm_fp4(a, sa, b, sb, workspace=torch.empty(1024, dtype=torch.uint8, device=dev))


# ---------------------------------------------------------------------------
# padded batches, uneven loads, strides, arguments that exclude each other


@pytest.mark.parametrize("T", [4, 300])
def test_padded_batch_under_the_debug_check(gpu_lib, monkeypatch, T):
    """Unrouted tokens leave rows behind the last expert's: the products take
    offsets that end below M_total, with MX_DEBUG too, and keep those rows of C."""
    mx = gpu_lib
    E, k, H, F = 8, 2, 256, 256
    x = mxsynth.normal_bf16((T, H), 1.0, seed=1).to(dev)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(2)).to(dev)
    mask = torch.ones(T, dtype=torch.bool, device=dev)
    mask[T // 2:] = False
    logits[~mask], x[~mask] = float("nan"), float("nan")
    W = _weights(mx, E, H, F, 5)
    want, f = _forward(mx, x, logits, W, E, k, mask=mask)
    n = int(f["off"][-1])
    assert n == T // 2 * k
    monkeypatch.setenv("MX_DEBUG", "1")
    o = dict(gu=torch.full((T * k, 2 * F), 7.0, dtype=torch.bfloat16, device=dev),
             y=torch.full((T * k, H), 7.0, dtype=torch.bfloat16, device=dev))
    out, f = _forward(mx, x, logits, W, E, k, o=o, mask=mask)
    assert torch.equal(out, want) and (out[~mask] == 0).all() and torch.isfinite(out).all()
    assert (f["gu"][n:] == 7).all() and (f["y"][n:] == 7).all()
    b = _backward(mx, torch.ones_like(out), logits, f, W)
    assert (b["dx"][~mask] == 0).all() and torch.isfinite(b["dx"]).all() and torch.isfinite(b["dh"][:n]).all()
    # what the check is for is still refused
    for bad, at in (([1, 1, 2], 0), ([0, 2, 1], 1), ([0, 1, n + T * k], 2)):
        with pytest.raises(mx.MxError, match=rf"group_offsets\[{at}\]"):
            mx.mx_grouped_gemm_fp4(torch.tensor(bad, device=dev), f["q"], f["s"], W["gu"][0][:2].contiguous(), W["gu"][1])


def _takes_few_rows(G, M, N):
    """The rule by which a grouped product takes the few-row kernel."""
    live = min(G, M)
    return live * ((N + 127) // 128) < torch.cuda.get_device_properties(0).multi_processor_count and M <= 16 * live


def test_few_rows_of_experts_beyond_4_gib(gpu_lib):
    """The few-row kernel with an expert whose weights start beyond 2^32 bytes."""
    mx = gpu_lib
    g = torch.Generator(device=dev)
    g.manual_seed(8)
    G, N, K = 260, 8192, 4096
    rows = [1, 2]
    m = sum(rows)
    assert _takes_few_rows(G, m, N)
    b, sb = _random_operand(g, G * N, K)
    assert (G - 1) * N * K // 2 > 1 << 32
    a, sa = _random_operand(g, m, K)
    off = torch.full((G + 1,), rows[0], dtype=torch.int64, device=dev)
    off[0], off[G] = 0, m
    C = mx.mx_grouped_gemm_fp4(off, a, sa, b.view(G, N, K // 2), sb)
    A, per = _decode(a, sa), N * K // 32
    for e, lo, hi in ((0, 0, rows[0]), (G - 1, rows[0], m)):
        _close(C[lo:hi], A[lo:hi], _decode(b[e * N:(e + 1) * N], sb[e * per:(e + 1) * per]), f"expert {e}")


@pytest.mark.parametrize("rows,N,K", [
    ([17, 0, 30, 1, 16, 0, 64, 0], 3968, 4096),      # chunks of 17 to 64 rows, long K
    ([0, 128, 0, 0, 0, 0, 0, 0], 3968, 4096),        # every row on one expert: two chunks
    ([33, 95, 0, 0, 0, 0, 0, 0], 2048, 14336), ([0, 0, 0, 0, 0, 0, 0, 120], 1000, 12288),
    ([15, 32, 33, 0, 48, 0, 0, 0], 130, 8192)])
def test_few_rows_of_uneven_loads(gpu_lib, rows, N, K):
    """Chunks of several passes of 16 rows, and more of K than stays in registers."""
    mx = gpu_lib
    G, M = len(rows), sum(rows)
    assert _takes_few_rows(G, M, N)
    g = torch.Generator(device=dev)
    g.manual_seed(M + K)
    off = np.concatenate([[0], np.cumsum(rows)])
    a, sa = _random_operand(g, M, K)
    n32 = (N + 31) // 32 * 32
    b = torch.randint(0, 256, (G, N, K // 2), generator=g, device=dev, dtype=torch.uint8)
    sb = torch.randint(121, 134, (G, n32 * (K // 32)), generator=g, device=dev, dtype=torch.uint8)
    A = _decode(a, sa)
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.full((M + 1, N), 7.0, dtype=dt, device=dev)
        C = mx.mx_grouped_gemm_fp4(torch.from_numpy(off).to(dev), a, sa, b, sb, c=buf[:M])
        for e in range(G):
            if rows[e]:
                lo, hi = off[e], off[e + 1]
                _close(C[lo:hi], A[lo:hi], _decode(b[e], sb[e]), f"expert {e}")
        assert (buf[M] == 7).all()
        assert torch.equal(C, mx.mx_grouped_gemm_fp4(torch.from_numpy(off).to(dev), a, sa, b, sb, out_dtype=dt))


@pytest.mark.parametrize("M", [7, 290])
def test_strided_operands_give_the_same_bytes(gpu_lib, M):
    """The sums' order goes by M, N and K alone: operands and C of any stride
    and alignment give what contiguous ones do."""
    mx = gpu_lib
    g = torch.Generator(device=dev)
    g.manual_seed(M)
    N, K = 272, 1024
    a, sa = _random_operand(g, M, K)
    b, sb = _random_operand(g, N, K)
    wa = torch.full((M, K // 2 + 48), 0x77, dtype=torch.uint8, device=dev)
    wb = torch.full((N, K // 2 + 16), 0x77, dtype=torch.uint8, device=dev)
    wa[:, 16:16 + K // 2], wb[:, :K // 2] = a, b
    for dt in (torch.bfloat16, torch.float32):
        want = mx.mx_gemm_fp4(a, sa, b, sb, out_dtype=dt)
        for pad, left in ((0, 0), (8, 8), (5, 3), (1, 0)):
            buf = torch.full((M, N + left + pad), 9.0, dtype=dt, device=dev)
            mx.mx_gemm_fp4(wa[:, 16:16 + K // 2], sa, wb[:, :K // 2], sb, c=buf[:, left:left + N])
            assert torch.equal(buf[:, left:left + N], want)
            assert (buf[:, :left] == 9).all() and (buf[:, left + N:] == 9).all()


def test_combine_gradient_refuses_an_output_that_is_not_wanted(gpu_lib):
    mx = gpu_lib
    x = torch.randn(4, 256, device=dev).bfloat16()
    y = torch.randn(8, 256, device=dev).bfloat16()
    slot = torch.arange(8, dtype=torch.int32, device=dev)
    w = torch.rand(4, 2, device=dev)
    with pytest.raises(ValueError, match="dy"):
        mx.mx_moe_combine_bwd(x, y, slot, w, dy=torch.empty_like(y), want_dy=False)
    with pytest.raises(ValueError, match="d_weights"):
        mx.mx_moe_combine_bwd(x, y, slot, w, d_weights=torch.empty_like(w), want_d_weights=False)


@pytest.mark.parametrize("T", [6, 40, 700])
def test_captured_layer_replayed_on_new_inputs(gpu_lib, T):
    """One capture, replayed with other tokens, logits and masks written into
    its inputs: experts' loads change, from none to all rows on one expert."""
    mx = gpu_lib
    E, k, H, F = 8, 2, 512, 256
    W = _weights(mx, E, H, F, 5)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=dev)
    logits = torch.zeros(T, E, device=dev)
    mask = torch.ones(T, dtype=torch.uint8, device=dev)
    d_out = mxsynth.normal_bf16((T, H), 1e-2, seed=9).to(dev)
    ws = torch.empty(max(mx.mx_moe_dispatch_workspace_bytes(T, k, E), 1), dtype=torch.uint8, device=dev)
    o = _buffers(T, E, k, H, F)
    how = dict(renormalize=False)

    def run(out):
        _, f = _forward(mx, x, logits, W, E, k, o=out, ws=ws if out else None, mask=mask, **how)
        return f, _backward(mx, d_out, logits, f, W, o=out, **how)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        run(o)
    for rep in range(5):
        x.copy_(mxsynth.normal_bf16((T, H), 1.0, seed=20 + rep))
        logits.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(rep)))
        mask.fill_(1)
        if rep == 1:
            logits[:, 3], logits[:, 5] = 9.0, 8.0         # every row on two experts
        if rep == 2:
            mask.zero_()                                  # no token at all
            logits.fill_(float("nan"))
        if rep == 3:
            mask[T // 3:] = 0                             # padded, the padding's logits anything
            logits[T // 3:] = float("nan")
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in o.items()}
        f, b = run(None)
        torch.cuda.synchronize()
        n = int(f["off"][-1])
        assert n == int(mask.sum()) * k
        for name in ("ids", "w", "off", "slot"):
            assert torch.equal(got[name], f[name]), f"replay {rep}: {name}"
        for name in ("q", "gu", "hq", "h", "y"):
            assert torch.equal(got[name][:n], f[name][:n]), f"replay {rep}: {name}"
        assert torch.equal(got["dw"], b["dw"]) and torch.equal(got["dx"], b["dx"]), f"replay {rep}"
        assert torch.equal(got["dh"][:n], b["dh"][:n]) and torch.equal(got["dy"][:n], b["dy"][:n]), f"replay {rep}"
        assert torch.isfinite(got["dx"]).all() and (got["dx"][mask == 0] == 0).all()
