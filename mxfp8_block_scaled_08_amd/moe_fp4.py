"""Binding of the ABI's second part (``include/mxfp8_moe_fp4.h``): routing of
tokens to experts and its gradient, the gradient of the MoE combine, and MXFP4
quantization and products.

As in the package's other functions, outputs that are passed in are written in
place and the rest are new tensors.  Every tensor of a call lives on one
device; the call runs on that device, on its current stream or on ``stream``,
and what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import _OUT, MX_BF16, MX_F32, _check, _u8, load, mx_moe_dispatch_workspace_bytes

MX_SCORE_SOFTMAX, MX_SCORE_SIGMOID = 0, 1

_SCORES = {"softmax": MX_SCORE_SOFTMAX, "sigmoid": MX_SCORE_SIGMOID}
_i, _l, _f, _p = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
_ARGS = {
    "mx_moe_route": [_p, _i, _l, _l, _l, _p, _i, _l, _l, _l, _l, _i, _f, _p, _p, _p, _p],
    "mx_moe_route_bwd": [_p, _i, _l, _l, _l, _i, _l, _i, _f, _p, _p, _p, _l, _p],
    "mx_moe_combine_bwd": [_p, _l, _l, _l, _p, _l, _p, _p, _l, _p, _l, _p, _p],
    "mx_quantize_rowwise_fp4": [_p, _l, _l, _l, _p, _l, _p, _l, _p],
    "mx_quantize_colwise_fp4": [_p, _l, _l, _l, _l, _p, _l, _p, _p],
    "mx_dequantize_fp4": [_p, _l, _l, _l, _p, _l, _p, _l, _i, _p],
    "mx_moe_dispatch_fp4": [_p, _l, _l, _l, _p, _l, _l, _p, _p, _p, _p, _l, _p, _p, _l, _p],
    "mx_swiglu_quantize_fp4": [_p, _l, _l, _l, _p, _l, _p, _l, _p, _p],
    "mx_gemm_fp4": [_l, _l, _l, _p, _l, _p, _p, _l, _p, _p, _l, _i, _p, _l, _p],
    "mx_grouped_gemm_fp4": [_l, _l, _l, _l, _p, _p, _l, _p, _p, _p, _p, _l, _i, _p],
}
_fns = {}


def _fn(name: str):
    """The library's entry point, its argument types set on first use."""
    f = _fns.get(name)
    if f is None:
        f = getattr(load(), name)
        f.restype = ctypes.c_int
        f.argtypes = _ARGS[name]
        _fns[name] = f
    return f


def _call(name: str, dev: torch.device, *args) -> None:
    """The entry point on dev's current stream (dev is the current device).

    The raw stream handle is asked for directly: a torch.cuda.Stream object
    for it costs 2.8 us, more than the whole launch."""
    st = _fn(name)(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        _check(name, st)


_current = torch._C._cuda_getDevice


def _elsewhere(fn, args: dict):
    """fn with its own arguments again (args: its locals), its first tensor's
    device current and, where stream is given, that stream current, so that the
    work, and every tensor that the call allocates, belongs to it.

    (Each function comes here first if its tensors are not on the current
    device or a stream is given; a decorator took 0.4 us of every call.)"""
    name = next(iter(args))
    dev, stream = args.pop("dev"), args.pop("stream")
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    elif not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return fn(**args)


def _at(t: torch.Tensor, name: str, dev, dtype, shape) -> int:
    """Pointer of t, a contiguous tensor of dtype and shape on dev."""
    if t.dtype is dtype and t.device == dev and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, is on {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be a contiguous {list(shape)} tensor, got {list(t.shape)}")


def _rows(t: torch.Tensor, name: str, dev, rows: int, cols: int, dtype) -> Tuple[int, int]:
    """(pointer, leading dimension) of a [rows][cols] row-major view of dtype on dev."""
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, is on {t.device}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}][{cols}], got {list(t.shape)}")
    return _first_rows(t, name, rows, cols, dtype)


def _first_rows(t: torch.Tensor, name: str, rows: int, cols: int, dtype) -> Tuple[int, int]:
    """The same of the tensor that the device and the sizes were taken from."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.is_contiguous():
        return t.data_ptr(), cols
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D row-major view")
    return t.data_ptr(), t.stride(0) if rows > 1 else cols


def _out_at(t: Optional[torch.Tensor], name: str, dev, dtype, *shape) -> Tuple[torch.Tensor, int]:
    """(t, pointer) of an output of dtype and shape on dev, a new tensor if t is None.

    (Sizes as separate arguments, and no check of what was just made: 0.6 us
    an output less of a call's 8.)"""
    if t is None:
        t = torch.empty(*shape, dtype=dtype, device=dev)
        return t, t.data_ptr()
    return t, _at(t, name, dev, dtype, shape)


def _out_rows(t: Optional[torch.Tensor], name: str, dev, rows: int, cols: int, dtype) -> Tuple[torch.Tensor, int, int]:
    """(t, pointer, leading dimension) of a [rows][cols] output on dev, a new tensor if t is None."""
    if t is None:
        t = torch.empty(rows, cols, dtype=dtype, device=dev)
        return t, t.data_ptr(), cols
    return (t, *_rows(t, name, dev, rows, cols, dtype))


def _one_of(t: torch.Tensor, name: str, dtypes):
    """t's dtype, which must be among dtypes."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    return t.dtype


def _out_dtype(t: Optional[torch.Tensor], name: str, dtype: torch.dtype) -> torch.dtype:
    """The output's type: t's, or dtype where a new tensor is made; BF16 or FP32."""
    if t is not None:
        return _one_of(t, name, _OUT)
    if dtype not in _OUT:
        raise ValueError(f"out_dtype must be {' or '.join(map(str, _OUT))}, got {dtype}")
    return dtype


_U8 = torch.uint8
_LOGITS = {torch.bfloat16: MX_BF16, torch.float32: MX_F32}


def _score(score: str) -> int:
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return _SCORES[score]


def mx_moe_route(logits: torch.Tensor, topk: int, *, bias: Optional[torch.Tensor] = None, score: str = "softmax",
                 num_groups: int = 1, topk_groups: int = 1, group_top: int = 1, renormalize: bool = True,
                 scale: float = 1.0, mask: Optional[torch.Tensor] = None, topk_ids: Optional[torch.Tensor] = None,
                 weights: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """logits [tokens][num_experts] (BF16 or FP32) -> (topk_ids int32, weights
    float32, both [tokens][topk]): each token's experts by decreasing score and
    their weights, what mx_moe_dispatch and mx_moe_combine take.

    bias (float32 [num_experts]) is added for the selection only; with
    num_groups > 1 only the topk_groups groups whose group_top best scores sum
    highest are chosen from; mask (uint8 or bool [tokens]) keeps tokens with 0
    unrouted (ids -1, weights 0), as experts with a logit of -inf are."""
    dev = logits.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_moe_route, locals())
    tokens, experts = logits.shape
    dtype = _one_of(logits, "logits", _LOGITS)
    x, ld = _first_rows(logits, "logits", tokens, experts, dtype)
    pb = None if bias is None else _at(bias, "bias", dev, torch.float32, (experts,))
    pm = None if mask is None else _at(mask, "mask", dev, torch.bool if mask.dtype is torch.bool else _U8, (tokens,))
    score = _score(score)
    topk_ids, pi = _out_at(topk_ids, "topk_ids", dev, torch.int32, tokens, topk)
    weights, pw = _out_at(weights, "weights", dev, torch.float32, tokens, topk)
    _call("mx_moe_route", dev, x, _LOGITS[dtype], tokens, experts, ld, pb, score, num_groups, topk_groups, group_top,
          topk, int(renormalize), scale, pm, pi, pw)
    return topk_ids, weights


def mx_moe_route_bwd(d_weights: torch.Tensor, logits: torch.Tensor, topk_ids: torch.Tensor, *, score: str = "softmax",
                     renormalize: bool = True, scale: float = 1.0, d_logits: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """Gradient of mx_moe_route's weights with respect to the logits (the
    choice topk_ids held fixed): [tokens][num_experts] of the logits' type."""
    dev = d_weights.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_moe_route_bwd, locals())
    tokens, experts = logits.shape
    topk = topk_ids.shape[1]
    dtype = _one_of(logits, "logits", _LOGITS)
    x, ld = _rows(logits, "logits", dev, tokens, experts, dtype)
    pi = _at(topk_ids, "topk_ids", dev, torch.int32, (tokens, topk))
    pw = _at(d_weights, "d_weights", dev, torch.float32, (tokens, topk))
    score = _score(score)
    d_logits, d, ld_d = _out_rows(d_logits, "d_logits", dev, tokens, experts, dtype)
    _call("mx_moe_route_bwd", dev, x, _LOGITS[dtype], tokens, experts, ld, score, topk, int(renormalize), scale, pi, pw,
          d, ld_d)
    return d_logits


def mx_moe_combine_bwd(d_out: torch.Tensor, y: Optional[torch.Tensor], slot: torch.Tensor, weights: torch.Tensor,
                       dy: Optional[torch.Tensor] = None, d_weights: Optional[torch.Tensor] = None,
                       want_dy: bool = True, want_d_weights: bool = True,
                       stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of mx_moe_combine: (dy BF16 [tokens*topk][hidden], d_weights
    float32 [tokens][topk]); either can be left out (then y may be None without
    d_weights).  Rows of dy that no slot names are not written (a new dy holds
    zeros there: it is cleared first, which at 20480 tokens x 8 x 2048 adds 105
    us to the call's 268; a dy that is passed in is not)."""
    dev = d_out.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_moe_combine_bwd, locals())
    tokens, topk = weights.shape
    hidden = d_out.shape[1]
    n = tokens * topk
    bf = torch.bfloat16
    if want_d_weights and y is None:
        raise ValueError("d_weights needs y")
    if (dy is not None and not want_dy) or (d_weights is not None and not want_d_weights):
        raise ValueError("dy or d_weights is given but not wanted")
    o, ld_o = _rows(d_out, "d_out", dev, tokens, hidden, bf)
    py, ld_y = _rows(y, "y", dev, n, hidden, bf) if want_d_weights else (None, 0)
    if slot.shape != (n,) and slot.shape != (tokens, topk):
        raise ValueError(f"slot must hold {n} entries, got {list(slot.shape)}")
    ps = _at(slot, "slot", dev, torch.int32, slot.shape)
    pw = _at(weights, "weights", dev, torch.float32, (tokens, topk))
    pd, ld_dy, pg = None, 0, None
    if want_dy:
        if dy is None:
            dy = torch.zeros((n, hidden), dtype=bf, device=dev)
        pd, ld_dy = _rows(dy, "dy", dev, n, hidden, bf)
    if want_d_weights:
        d_weights, pg = _out_at(d_weights, "d_weights", dev, torch.float32, tokens, topk)
    _call("mx_moe_combine_bwd", dev, o, tokens, hidden, ld_o, py, ld_y, ps, pw, topk, pd, ld_dy, pg)
    return dy if want_dy else None, d_weights if want_d_weights else None


def _scale_ptr(s: torch.Tensor, name: str, dev, need: int) -> int:
    """Pointer of a rearranged scale buffer on dev of at least need bytes."""
    if s.dtype is not _U8:
        s = _u8(s)
    if s.dtype is _U8 and s.device == dev and s.numel() >= need and s.is_contiguous():
        return s.data_ptr()
    raise ValueError(f"{name} must be a contiguous uint8 tensor of at least {need} bytes on {dev}, got {s.numel()} of "
                     f"{s.dtype} on {s.device}")


def _scale_bytes(rows: int, cols: int, tiles: int) -> int:
    """Bytes from the first to the last tile of [rows][cols/32] scales, `tiles` tiles a tile row."""
    return ((rows + 31) // 32 * tiles - tiles + cols // 256) * 256 if rows and cols else 0


def _scales(s: Optional[torch.Tensor], rows: int, cols: int, tiles: int, name: str, dev):
    """(tensor, pointer) of rearranged scales to write (a new buffer if None)."""
    if s is None and tiles >= cols // 256:
        s = torch.empty(max((rows + 31) // 32 * tiles * 256, 1), dtype=_U8, device=dev)
        return s, s.data_ptr()
    if s is None:
        raise ValueError(f"s_tiles={tiles} is less than the {cols // 256} tiles of a row")
    return s, _scale_ptr(s, name, dev, _scale_bytes(rows, cols, tiles))


def mx_quantize_rowwise_fp4(x: torch.Tensor, q: Optional[torch.Tensor] = None, s_swz: Optional[torch.Tensor] = None,
                            s_tiles: Optional[int] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """BF16 x[rows][cols] -> (q uint8 [rows][cols/2] E2M1, two codes a byte,
    s_swz: its scales in the products' layout)."""
    dev = x.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_quantize_rowwise_fp4, locals())
    rows, cols = x.shape
    px, ld_x = _first_rows(x, "x", rows, cols, torch.bfloat16)
    if s_tiles is None:
        s_tiles = cols // 256
    q, pq, ld_q = _out_rows(q, "q", dev, rows, cols // 2, _U8)
    s_swz, ps = _scales(s_swz, rows, cols, s_tiles, "s_swz", dev)
    _call("mx_quantize_rowwise_fp4", dev, px, rows, cols, ld_x, pq, ld_q, ps, s_tiles)
    return q, s_swz


def mx_quantize_colwise_fp4(x: torch.Tensor, qt: Optional[torch.Tensor] = None, st_swz: Optional[torch.Tensor] = None,
                            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """BF16 x [rows][cols], or a stack [count][rows][cols] -> (qt uint8
    [(count][)cols][rows/2], st_swz): each tensor quantized down its columns and
    written transposed, the stack's scales back to back."""
    dev = x.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_quantize_colwise_fp4, locals())
    bf = torch.bfloat16
    if x.dim() == 3:
        count, rows, cols = x.shape
        if not x.is_contiguous():
            raise ValueError("a stack must be contiguous [count][rows][cols]")
        px, ld_x = _first_rows(x, "x", count * rows, cols, bf)
        qt, pq = _out_at(qt, "qt", dev, _U8, count, cols, rows // 2)
        ld_qt = rows // 2
    else:
        (rows, cols), count = x.shape, 1
        px, ld_x = _first_rows(x, "x", rows, cols, bf)
        qt, pq, ld_qt = _out_rows(qt, "qt", dev, cols, rows // 2, _U8)
    need = count * _scale_bytes(cols, rows, rows // 256)
    if st_swz is None:
        st_swz = torch.empty(max(need, 1), dtype=_U8, device=dev)
    _call("mx_quantize_colwise_fp4", dev, px, count, rows, cols, ld_x, pq, ld_qt,
          _scale_ptr(st_swz, "st_swz", dev, need))
    return qt, st_swz


def mx_dequantize_fp4(q: torch.Tensor, s_swz: torch.Tensor, y: Optional[torch.Tensor] = None,
                      out_dtype: torch.dtype = torch.bfloat16, s_tiles: Optional[int] = None,
                      stream=None) -> torch.Tensor:
    """The values of an MXFP4 operand (q [rows][cols/2], rearranged scales) as
    BF16 or FP32 [rows][cols]; exact in both."""
    dev = q.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_dequantize_fp4, locals())
    rows, half = q.shape
    cols = 2 * half
    if s_tiles is None:
        s_tiles = cols // 256
    pq, ld_q = _first_rows(q, "q", rows, half, _U8)
    ps = _scale_ptr(s_swz, "s_swz", dev, _scale_bytes(rows, cols, s_tiles))
    y, py, ld_y = _out_rows(y, "y", dev, rows, cols, _out_dtype(y, "y", out_dtype))
    _call("mx_dequantize_fp4", dev, pq, rows, cols, ld_q, ps, s_tiles, py, ld_y, _OUT[y.dtype])
    return y


def mx_moe_dispatch_fp4(x: torch.Tensor, topk_ids: torch.Tensor, num_experts: int,
                        offsets: Optional[torch.Tensor] = None, src: Optional[torch.Tensor] = None,
                        slot: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                        s_swz: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """mx_moe_dispatch with MXFP4 rows: (offsets, src_token, slot, q uint8
    [tokens*topk][hidden/2], s_swz)."""
    dev = x.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_moe_dispatch_fp4, locals())
    tokens, hidden = x.shape
    if topk_ids.dim() != 2 or topk_ids.shape[0] != tokens:
        raise ValueError("topk_ids must be [tokens][topk]")
    topk = topk_ids.shape[1]
    n = tokens * topk
    i32 = torch.int32
    px, ld_x = _first_rows(x, "x", tokens, hidden, torch.bfloat16)
    pi = _at(topk_ids, "topk_ids", dev, i32, (tokens, topk))
    offsets, po = _out_at(offsets, "offsets", dev, torch.int64, num_experts + 1)
    src, pr = _out_at(src, "src", dev, i32, n)
    slot, pl = _out_at(slot, "slot", dev, i32, n)
    q, pq, ld_q = _out_rows(q, "q", dev, n, hidden // 2, _U8)
    s_swz, ps = _scales(s_swz, n, hidden, hidden // 256, "s_swz", dev)
    if workspace is None:
        workspace = torch.empty(max(mx_moe_dispatch_workspace_bytes(tokens, topk, num_experts), 1), dtype=_U8, device=dev)
    pw, nw = _scratch(workspace, dev)
    _call("mx_moe_dispatch_fp4", dev, px, tokens, hidden, ld_x, pi, topk, num_experts, po, pr, pl, pq, ld_q, ps, pw, nw)
    return offsets, src, slot, q, s_swz


def _scratch(workspace: Optional[torch.Tensor], dev) -> Tuple[Optional[int], int]:
    if workspace is None:
        return None, 0
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def mx_swiglu_quantize_fp4(gu: torch.Tensor, q: Optional[torch.Tensor] = None, s_swz: Optional[torch.Tensor] = None,
                           h: Optional[torch.Tensor] = None, want_h: bool = False, stream=None):
    """gu [rows][2F] BF16 (gate | up) -> (q uint8 [rows][F/2], s_swz, h or
    None): mx_swiglu_quantize with MXFP4 output."""
    dev = gu.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_swiglu_quantize_fp4, locals())
    rows, F2 = gu.shape
    F = F2 // 2
    pg, ld_gu = _first_rows(gu, "gu", rows, F2, torch.bfloat16)
    ph, ld_h = None, 0
    if h is not None or want_h:
        h, ph, ld_h = _out_rows(h, "h", dev, rows, F, torch.bfloat16)
    q, pq, ld_q = _out_rows(q, "q", dev, rows, F // 2, _U8)
    s_swz, ps = _scales(s_swz, rows, F, F // 256, "s_swz", dev)
    _call("mx_swiglu_quantize_fp4", dev, pg, rows, F, ld_gu, ph, ld_h, pq, ld_q, ps)
    return q, s_swz, h


def mx_gemm_fp4_workspace_bytes(M: int, N: int, K: int, out_dtype: torch.dtype = torch.bfloat16) -> int:
    """Device scratch mx_gemm_fp4 needs for this shape (0: none), host-only."""
    f = _fns.get("mx_gemm_fp4_workspace_bytes")
    if f is None:
        f = load().mx_gemm_fp4_workspace_bytes
        f.restype, f.argtypes = ctypes.c_int64, [_l, _l, _l, _i]
        _fns["mx_gemm_fp4_workspace_bytes"] = f
    return f(M, N, K, _OUT[out_dtype])


@functools.lru_cache(maxsize=1024)
def _gemm_workspace(device: int, M: int, N: int, K: int, dtype: torch.dtype) -> int:
    """mx_gemm_fp4_workspace_bytes on the current device, which is `device`: a
    function of the shape and the device alone."""
    return mx_gemm_fp4_workspace_bytes(M, N, K, dtype)


def mx_gemm_fp4(a_q: torch.Tensor, a_s_swz: torch.Tensor, b_q: torch.Tensor, b_s_swz: torch.Tensor,
                c: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """C[M][N] = deq(A) . deq(B)^T for MXFP4 operands A [M][K/2 bytes], B
    [N][K/2 bytes].  workspace: device scratch of at least
    mx_gemm_fp4_workspace_bytes bytes when that is nonzero (a new tensor if
    None)."""
    dev = a_q.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_gemm_fp4, locals())
    M, half = a_q.shape
    N, K = b_q.shape[0], 2 * half
    pa, ld_a = _first_rows(a_q, "a_q", M, half, _U8)
    pb, ld_b = _rows(b_q, "b_q", dev, N, half, _U8)
    pas = _scale_ptr(a_s_swz, "a_s_swz", dev, _scale_bytes(M, K, K // 256))
    pbs = _scale_ptr(b_s_swz, "b_s_swz", dev, _scale_bytes(N, K, K // 256))
    dtype = _out_dtype(c, "c", out_dtype)
    c, pc, ld_c = _out_rows(c, "c", dev, M, N, dtype)
    if workspace is None:
        need = _gemm_workspace(dev.index, M, N, K, dtype)
        if need:
            workspace = torch.empty(need, dtype=_U8, device=dev)
    pw, nw = _scratch(workspace, dev)
    _call("mx_gemm_fp4", dev, M, N, K, pa, ld_a, pas, pb, ld_b, pbs, pc, ld_c, _OUT[dtype], pw, nw)
    return c


def mx_grouped_gemm_fp4(group_offsets: torch.Tensor, a_q: torch.Tensor, a_s_swz: torch.Tensor, b_q: torch.Tensor,
                        b_s_swz: torch.Tensor, c: Optional[torch.Tensor] = None,
                        out_dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """Per-expert C: rows [off[g], off[g+1]) of A times B_g^T, B as
    [G][N][K/2 bytes], MXFP4.  off[G] may be less than A's rows (unrouted
    assignments); rows outside every group are not written."""
    dev = group_offsets.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_grouped_gemm_fp4, locals())
    M, half = a_q.shape
    G, N, _ = b_q.shape
    K = 2 * half
    po = _at(group_offsets, "group_offsets", dev, torch.int64, (G + 1,))
    pa, ld_a = _rows(a_q, "a_q", dev, M, half, _U8)
    pas = _scale_ptr(a_s_swz, "a_s_swz", dev, _scale_bytes(M, K, K // 256))
    pb = _at(b_q, "b_q", dev, _U8, (G, N, half))
    pbs = _scale_ptr(b_s_swz, "b_s_swz", dev, G * ((N + 31) // 32) * K)
    dtype = _out_dtype(c, "c", out_dtype)
    c, pc, ld_c = _out_rows(c, "c", dev, M, N, dtype)
    _call("mx_grouped_gemm_fp4", dev, G, M, N, K, po, pa, ld_a, pas, pb, pbs, pc, ld_c, _OUT[dtype])
    return c
