"""CPU checks of the ABI's second part (include/mxfp8_moe_fp4.h): every
declared entry point is exported and bound, and invalid arguments are refused
before HIP is touched (fake pointers are never dereferenced)."""
import ctypes
import inspect
import math
import os
import re

import numpy as np
import pytest
import torch

import fp4_ref as ref
import mxfp8_block_scaled_08_amd as mx
import mxsynth
from mxfp8_block_scaled_08_amd import moe_fp4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D, E, F, G = (i << 32 for i in range(1, 8))
BF, F32 = mx.MX_BF16, mx.MX_F32
INV, SHAPE, ALIGN, OVER, UNSUP = (mx.MX_ERR_INVALID_ARG, mx.MX_ERR_SHAPE, mx.MX_ERR_ALIGN, mx.MX_ERR_OVERLAP,
                                  mx.MX_ERR_UNSUPPORTED)


def call(name, base, **kw):
    """The entry point with arguments base (a dict in order), some replaced."""
    args = dict(base)
    assert set(kw) <= set(args)
    args.update(kw)
    return moe_fp4._fn(name)(*args.values(), None)


def refused(name, base, status, word="", **kw):
    assert call(name, base, **kw) == status, mx.mx_last_error()
    assert name in mx.mx_last_error() and word in mx.mx_last_error()


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxfp8_moe_fp4.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mx_[a-z_0-9]+)\s*\(", text)))
    assert len(names) == 11
    raw = ctypes.CDLL(mx.lib_path())
    for n in names:
        assert hasattr(raw, n) and hasattr(mx, n) and n in mx.__all__, n
        if n in moe_fp4._ARGS:
            decl = re.search(n + r"\s*\((.*?)\)\s*;", text, flags=re.S).group(1)
            assert len(moe_fp4._ARGS[n]) == decl.count(",") + 1, n
            assert "stream" in inspect.signature(getattr(mx, n)).parameters, n


ROUTE = dict(logits=A, dt=F32, tokens=4, experts=64, ld=64, bias=B, score=0, groups=1, keep=1, gtop=1, topk=8, renorm=1,
             scale=1.0, mask=None, ids=C, w=D)


def test_route_refusals():
    r = lambda st, word="", **kw: refused("mx_moe_route", ROUTE, st, word, **kw)  # noqa: E731
    r(INV, "logits_dtype", dt=2)
    r(INV, "score", score=2)
    r(INV, tokens=-1)
    r(INV, experts=0)
    r(INV, topk=0)
    r(UNSUP, "num_experts", experts=1025, ld=1025)
    r(UNSUP, "topk", topk=33)
    r(INV, "leading", ld=63)
    r(INV, "scale", scale=math.inf)
    r(INV, "scale", scale=math.nan)
    r(INV, "num_groups", groups=7)
    r(INV, "num_groups", groups=0)
    r(INV, "num_groups", groups=8, keep=9)
    r(INV, "num_groups", groups=8, keep=0)
    r(UNSUP, "num_groups", groups=128, keep=128, experts=256, ld=256)
    r(INV, "group_top", gtop=3)
    r(INV, "group_top", groups=64, keep=64, gtop=2)
    r(INV, "topk", groups=32, keep=2, gtop=1)
    r(INV, "topk", experts=7, ld=7)
    r(INV, "null", logits=None)
    r(INV, "null", ids=None)
    r(INV, "null", w=None)
    r(ALIGN, logits=A + 2)
    r(ALIGN, bias=B + 1)
    r(ALIGN, ids=C + 2)
    r(ALIGN, w=D + 2)
    r(OVER, ids=A + 64)
    r(OVER, w=C + 4)
    r(OVER, w=B)
    r(OVER, mask=C + 3)
    r(UNSUP, tokens=1 << 31)
    assert call("mx_moe_route", ROUTE, tokens=0) == mx.MX_OK


def test_route_bwd_refusals():
    base = dict(logits=A, dt=BF, tokens=4, experts=64, ld=64, score=1, topk=8, renorm=1, scale=1.0, ids=B, dw=C, dx=D,
                ld_d=64)
    r = lambda st, word="", **kw: refused("mx_moe_route_bwd", base, st, word, **kw)  # noqa: E731
    r(INV, dt=7)
    r(INV, score=-1)
    r(INV, "ld_d", ld_d=63)
    r(UNSUP, topk=40)
    r(INV, "null", dw=None)
    r(INV, "null", dx=None)
    r(ALIGN, dx=D + 1)
    r(OVER, dx=A + 2)
    r(OVER, dx=B)
    r(OVER, dx=C + 8)
    assert call("mx_moe_route_bwd", base, tokens=0) == mx.MX_OK


def test_combine_bwd_refusals():
    base = dict(d_out=A, tokens=4, hidden=64, ld_o=64, y=B, ld_y=64, slot=C, w=D, topk=2, dy=E, ld_dy=64, dw=F)
    r = lambda st, word="", **kw: refused("mx_moe_combine_bwd", base, st, word, **kw)  # noqa: E731
    r(INV, tokens=-1)
    r(INV, topk=0)
    r(SHAPE, "hidden", hidden=60)
    r(INV, "2^30", tokens=1 << 29, topk=4)
    r(INV, "leading", ld_o=56)
    r(INV, "leading", ld_y=56)
    r(INV, "leading", ld_dy=56)
    r(INV, "null", y=None)
    r(INV, "null", slot=None)
    r(INV, "null", d_out=None)
    r(ALIGN, y=B + 8)
    r(ALIGN, dy=E + 8)
    r(ALIGN, ld_o=68)
    r(ALIGN, dw=F + 2)
    r(OVER, dy=B + 64)
    r(OVER, dw=E)
    r(OVER, dw=C)
    assert call("mx_moe_combine_bwd", base, tokens=0) == mx.MX_OK
    assert call("mx_moe_combine_bwd", base, dy=None, dw=None) == mx.MX_OK


def test_quantize_refusals():
    row = dict(x=A, rows=4, cols=256, ld_x=256, q=B, ld_q=128, s=C, tiles=1)
    r = lambda st, word="", **kw: refused("mx_quantize_rowwise_fp4", row, st, word, **kw)  # noqa: E731
    r(INV, rows=-1)
    r(SHAPE, cols=250)
    r(UNSUP, cols=128)
    r(INV, ld_x=248)
    r(INV, ld_q=112)
    r(INV, tiles=0)
    r(INV, "null", s=None)
    r(ALIGN, x=A + 8)
    r(ALIGN, q=B + 4)
    r(ALIGN, ld_x=260)
    r(ALIGN, ld_q=136)
    r(OVER, q=A + 256)
    r(OVER, s=B + 128)
    r(UNSUP, rows=1 << 33)
    assert call("mx_quantize_rowwise_fp4", row, rows=0) == mx.MX_OK
    col = dict(x=A, count=2, rows=256, cols=64, ld_x=64, qt=B, ld_qt=128, scales=C)
    r = lambda st, word="", **kw: refused("mx_quantize_colwise_fp4", col, st, word, **kw)  # noqa: E731
    r(INV, count=-1)
    r(SHAPE, rows=250)
    r(SHAPE, cols=40, ld_x=40)
    r(UNSUP, rows=128)
    r(INV, ld_x=56)
    r(INV, ld_qt=112)
    r(INV, "null", x=None)
    r(ALIGN, ld_x=66)
    r(ALIGN, qt=B + 8)
    r(ALIGN, scales=C + 2)
    r(OVER, qt=A + 32)
    r(OVER, scales=B + 16 * 64)
    r(UNSUP, count=1 << 40)
    r(UNSUP, rows=1 << 25, cols=1 << 25, ld_x=1 << 25, ld_qt=1 << 24)      # 2^36 tiles
    assert call("mx_quantize_colwise_fp4", col, count=0) == mx.MX_OK
    deq = dict(q=A, rows=4, cols=256, ld_q=128, s=B, tiles=1, y=C, ld_y=256, dt=BF)
    r = lambda st, word="", **kw: refused("mx_dequantize_fp4", deq, st, word, **kw)  # noqa: E731
    r(INV, "y_dtype", dt=2)
    r(INV, ld_y=248)
    r(UNSUP, cols=32)
    r(ALIGN, ld_y=260)
    r(ALIGN, y=C + 4)
    r(ALIGN, q=A + 8)
    r(OVER, y=A)
    r(OVER, y=B)
    r(INV, "null", y=None)


def test_dispatch_and_swiglu_refusals():
    dis = dict(x=A, tokens=4, hidden=256, ld_x=256, ids=B, topk=2, experts=8, off=C, src=D, slot=E, q=F, ld_q=128, s=G,
               ws=8 << 32, wsb=1 << 20)
    r = lambda st, word="", **kw: refused("mx_moe_dispatch_fp4", dis, st, word, **kw)  # noqa: E731
    r(INV, tokens=0)
    r(INV, experts=0)
    r(UNSUP, experts=2000)
    r(UNSUP, tokens=1 << 30)
    r(SHAPE, hidden=250)
    r(UNSUP, hidden=128)
    r(INV, hidden=0)
    r(INV, ld_q=64)
    r(INV, "null", slot=None)
    r(ALIGN, off=C + 4)
    r(OVER, slot=D)
    r(INV, "workspace", wsb=8)
    r(ALIGN, "workspace", ws=(8 << 32) + 2)
    r(OVER, "workspace", ws=F + 64)
    sw = dict(gu=A, rows=4, f=256, ld_gu=512, h=None, ld_h=0, q=B, ld_q=128, s=C)
    r = lambda st, word="", **kw: refused("mx_swiglu_quantize_fp4", sw, st, word, **kw)  # noqa: E731
    r(INV, ld_gu=256)
    r(INV, h=D, ld_h=200)
    r(UNSUP, f=32)
    r(ALIGN, h=D + 2, ld_h=256)
    r(OVER, h=A, ld_h=256)
    r(INV, "null", gu=None)
    assert call("mx_swiglu_quantize_fp4", sw, rows=0) == mx.MX_OK


def test_gemm_refusals():
    g = dict(M=100, N=64, K=512, a=A, ld_a=256, a_s=B, b=C, ld_b=256, b_s=D, c=E, ld_c=64, dt=BF, ws=F, wsb=1 << 26)
    r = lambda st, word="", **kw: refused("mx_gemm_fp4", g, st, word, **kw)  # noqa: E731
    r(INV, M=-1)
    r(INV, dt=3)
    r(SHAPE, K=0)
    r(SHAPE, K=40)
    r(UNSUP, K=128)
    r(INV, ld_a=128)
    r(INV, ld_b=128)
    r(INV, ld_c=63)
    r(INV, "null", b_s=None)
    r(ALIGN, a=A + 8)
    r(ALIGN, ld_b=264)
    r(ALIGN, a_s=B + 2)
    r(ALIGN, c=E + 1)
    r(OVER, c=A)
    r(OVER, c=D)
    r(UNSUP, ld_a=1 << 24)
    r(UNSUP, ld_c=1 << 24)
    r(INV, "workspace", wsb=-1)
    assert call("mx_gemm_fp4", g, M=0) == mx.MX_OK
    gg = dict(G=4, M=100, N=64, K=512, off=F, a=A, ld_a=256, a_s=B, b=C, b_s=D, c=E, ld_c=64, dt=F32)
    r = lambda st, word="", **kw: refused("mx_grouped_gemm_fp4", gg, st, word, **kw)  # noqa: E731
    r(INV, G=0)
    r(UNSUP, G=1025)
    r(INV, "group_offsets", off=None)
    r(ALIGN, off=F + 4)
    r(OVER, c=F)
    r(OVER, c=C + 512)
    r(UNSUP, K=384)
    r(INV, ld_c=60)
    assert call("mx_grouped_gemm_fp4", gg, M=0) == mx.MX_OK


def test_limits_of_sizes():
    """Sizes at the stated limits: the largest that is taken reaches the checks behind it."""
    combine = dict(d_out=A, tokens=4, hidden=64, ld_o=64, y=B, ld_y=64, slot=None, w=D, topk=2, dy=E, ld_dy=64, dw=F)
    for tokens, topk in ((1 << 29, 2), (1 << 30, 1), (1, 1 << 30), (1 << 27, 8)):
        refused("mx_moe_combine_bwd", combine, INV, "2^30", tokens=tokens, topk=topk)
    for tokens, topk in (((1 << 29) - 1, 2), ((1 << 30) - 1, 1), (1, (1 << 30) - 1), (357913941, 3)):
        refused("mx_moe_combine_bwd", combine, INV, "null", tokens=tokens, topk=topk)
    # a launch of 2^32 threads, 64 a token, is one too many
    bwd = dict(logits=None, dt=BF, tokens=4, experts=1024, ld=1024, score=1, topk=8, renorm=1, scale=1.0, ids=B, dw=C,
               dx=D, ld_d=1024)
    for name, base in (("mx_moe_route", dict(ROUTE, logits=None)), ("mx_moe_route_bwd", bwd)):
        for tokens in ((1 << 26) - 3, (1 << 26) - 1, 1 << 26):
            refused(name, base, UNSUP, "tokens", tokens=tokens)
        refused(name, base, INV, "null", tokens=(1 << 26) - 4)
    refused("mx_moe_route", ROUTE, UNSUP, "leading", ld=1 << 28)
    refused("mx_moe_route_bwd", bwd, UNSUP, "leading", ld=1 << 28)
    refused("mx_moe_route_bwd", bwd, UNSUP, "ld_d", ld_d=1 << 28)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 16)
    for f, args in ((mx.mx_moe_route, (x, 2)), (mx.mx_quantize_rowwise_fp4, (x,)), (mx.mx_gemm_fp4, (x, x, x, x))):
        with pytest.raises(ValueError):
            f(*args)


def test_reference_rounds_to_the_nearest_value():
    """The reference itself, against a search over all sixteen values."""
    rng = np.random.default_rng(0)
    bits = mxsynth.bits(mxsynth.normal_bf16((64, 256), 1.0, seed=1, outlier_frac=0.05, outlier_mul=30.0)).copy()
    bits[0, :32] = 0
    bits[1] = rng.integers(0, 128, 256)
    codes, scales = ref.quantize(bits)
    v = ref.bf16_values(bits)
    s = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)
    d = np.abs(np.abs(v)[..., None] / s[..., None] - ref.E2M1)
    got = np.abs(np.abs(v) / s - ref.E2M1[codes & 7])
    assert (got == d.min(-1)).all()
    ties = (d == d.min(-1, keepdims=True)).sum(-1) > 1
    assert ties.any() and ((codes & 7)[ties] % 2 == 0).all()
    amax = np.abs(v).reshape(64, 8, 32).max(-1) / np.ldexp(1.0, scales.astype(int) - 127)
    assert (((amax >= 4) & (amax < 8)) | (scales == 0)).all()
