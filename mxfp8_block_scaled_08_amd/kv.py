"""Binding of the ABI's third part (``include/mxfp8_kv.h``): rotary positions,
the paged 8-bit key/value cache and the attention over it.

A cache is two tensors and the call's sequences three:
  kv          uint8 [2 (K, V)][num_pages][kv_heads][page_size][head_dim], E4M3
              codes; any strides with rows of head_dim together
  kv_scale    uint8 [2][num_pages][kv_heads][page_size / 16], E8M0, contiguous
  page_table  int32 [batch][max_pages]
  kv_lens     int32 [batch], positions of a sequence, this call's rows included
  seq_starts  int64 [batch + 1]: rows seq_starts[b] .. seq_starts[b+1] - 1 are
              sequence b's and stand at its last positions
As in the package's other functions, outputs that are passed in are written in
place and the rest are new tensors; every tensor of a call lives on one device,
and the call runs there, on its current stream or on ``stream``.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional, Tuple

import torch

from . import MX_BF16, MX_F32, _check, load
from .moe_fp4 import _at, _current, _elsewhere, _one_of, _out_at, _scratch

MX_ROPE_HALF, MX_ROPE_INTERLEAVED = 0, 1
MX_ROPE_PLAIN, MX_ROPE_LINEAR, MX_ROPE_NTK, MX_ROPE_YARN, MX_ROPE_YARN_PAIRS = 0, 1, 2, 3, 4
MX_KV_BLOCK = 16

_STYLES = {"half": MX_ROPE_HALF, "interleaved": MX_ROPE_INTERLEAVED}
_SCALINGS = {"plain": MX_ROPE_PLAIN, "linear": MX_ROPE_LINEAR, "ntk": MX_ROPE_NTK, "yarn": MX_ROPE_YARN,
             "yarn_pairs": MX_ROPE_YARN_PAIRS}
_TYPES = {torch.bfloat16: MX_BF16, torch.float32: MX_F32}
_BF, _U8, _I32, _I64, _F64 = torch.bfloat16, torch.uint8, torch.int32, torch.int64, torch.float64
_i, _l, _f, _d, _p = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double, ctypes.c_void_p


class _Cache(ctypes.Structure):
    """mx_kv_cache.  (The calls pass the same 16 words as bytes: packing them takes
    0.6 us, filling the structure 1.6.)"""
    _fields_ = [("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p), ("num_pages", _l), ("kv_heads", _l),
                ("page_size", _l), ("head_dim", _l), ("ld_page", _l), ("ld_head", _l), ("ld_token", _l),
                ("page_table", _p), ("max_pages", _l), ("kv_lens", _p), ("seq_starts", _p), ("batch", _l)]


_pack = struct.Struct("=16q").pack
_ARGS = {
    "mx_rope_frequencies": [_l, _d, _i, _d, _l, _p, _p],
    "mx_rope": [_p, _i, _l, _l, _l, _l, _l, _p, _p, _l, _i, _f, _i, _p, _l, _l, _p],
    "mx_kv_append": [_p, _p, _l, _l, _p, _l, _l, _l, _p, _l, _i, _f, _p],
    "mx_kv_read": [_p, _l, _p, _p, _i, _p],
    "mx_kv_attention_workspace_bytes": [_l, _l, _l, _l, _l, _l],
    "mx_kv_attention": [_p, _p, _l, _l, _l, _l, _f, _i, _l, _l, _p, _l, _l, _p, _p, _l, _p],
}
_fns = {}


def _fn(name: str):
    """The library's entry point, its argument types set on first use."""
    f = _fns.get(name)
    if f is None:
        f = getattr(load(), name)
        f.restype = _l if name.endswith("_bytes") else _i
        f.argtypes = _ARGS[name]
        _fns[name] = f
    return f


def _call(name: str, dev: torch.device, *args) -> None:
    """The entry point on dev's current stream (dev is the current device)."""
    st = _fn(name)(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        _check(name, st)


def _style(style: str) -> int:
    if style not in _STYLES:
        raise ValueError(f"style must be 'half' or 'interleaved', got {style!r}")
    return _STYLES[style]


def _heads(t: torch.Tensor, name: str, dev, dtype, shape=None) -> Tuple[int, int, int]:
    """(pointer, stride of a row, stride of a head) of [rows][heads][dim] on dev, dim together."""
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, is on {t.device}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be {list(shape) if shape is not None else '[rows][heads][dim]'}, got {list(t.shape)}")
    s = t.stride()
    if s[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must hold a head's elements together")
    return t.data_ptr(), s[0], s[1]


def _cache(kv, kv_scale, page_table, kv_lens, seq_starts, dev) -> Tuple[bytes, int, int, int]:
    """(the call's mx_kv_cache, kv_heads, head_dim, batch)"""
    shape = kv.shape
    if len(shape) != 5 or shape[0] != 2 or kv.dtype is not _U8 or kv.device != dev:
        raise ValueError(f"kv must be uint8 [2][pages][kv_heads][page_size][head_dim] on {dev}, got {kv.dtype} "
                         f"{list(shape)} on {kv.device}")
    _, pages, heads, page, dim = shape
    both, s_page, s_head, s_token, one = kv.stride()
    if one != 1 and dim > 1:
        raise ValueError("kv must hold a row's codes together")
    scale = _at(kv_scale, "kv_scale", dev, _U8, (2, pages, heads, page // MX_KV_BLOCK))
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [batch][max_pages], got {list(page_table.shape)}")
    batch, most = page_table.shape
    k = kv.data_ptr()
    return _pack(k, k + both, scale, scale + pages * heads * (page // MX_KV_BLOCK), pages, heads, page, dim, s_page,
                 s_head, s_token, _at(page_table, "page_table", dev, _I32, (batch, most)), most,
                 _at(kv_lens, "kv_lens", dev, _I32, (batch,)),
                 _at(seq_starts, "seq_starts", dev, _I64, (batch + 1,)), batch), heads, dim, batch


def mx_rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                        original_len: int = 0, device="cuda") -> Tuple[torch.Tensor, float]:
    """(freqs float64 [rot_dim / 2] on device, amplitude): radians a position of
    every rotary pair, scaling 'plain', 'linear', 'ntk', 'yarn' or 'yarn_pairs'
    (include/mxfp8_kv.h).  For a checkpoint whose configuration names yarn scaling take
    'yarn_pairs', which ramps over the pairs' numbers; 'yarn' is the paper's formula,
    which ramps over the turns and gives other frequencies in between."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(_SCALINGS)}, got {scaling!r}")
    freqs = torch.empty(max(rot_dim // 2, 1), dtype=_F64)
    amplitude = ctypes.c_float()
    st = _fn("mx_rope_frequencies")(rot_dim, base, _SCALINGS[scaling], factor, original_len, freqs.data_ptr(),
                                    ctypes.addressof(amplitude))
    if st:
        _check("mx_rope_frequencies", st)
    return freqs.to(device), amplitude.value


def _rope(x, positions, freqs, style, amplitude, y, inverse: int, xn: str, yn: str) -> torch.Tensor:
    dev = x.device
    dtype = _one_of(x, xn, _TYPES)
    px, ld_xt, ld_xh = _heads(x, xn, dev, dtype)
    tokens, heads, dim = x.shape
    pp = _at(positions, "positions", dev, _I32, (tokens,))
    pf = _at(freqs, "freqs", dev, _F64, (freqs.numel(),))
    if y is None:
        y = torch.empty(tokens, heads, dim, dtype=dtype, device=dev)
        py, ld_yt, ld_yh = y.data_ptr(), heads * dim, dim
    else:
        py, ld_yt, ld_yh = _heads(y, yn, dev, dtype, x.shape)
    _call("mx_rope", dev, px, _TYPES[dtype], tokens, heads, dim, ld_xt, ld_xh, pp, pf, 2 * freqs.numel(), _style(style),
          amplitude, inverse, py, ld_yt, ld_yh)
    return y


def mx_rope(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, *, style: str = "half",
            amplitude: float = 1.0, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [tokens][heads][head_dim] (BF16 or FP32) turned by positions (int32
    [tokens]): pair i by positions[t] * freqs[i] radians, the first 2 * len(freqs)
    elements of a head; the rest is copied.  y may be x."""
    dev = x.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_rope, locals())
    return _rope(x, positions, freqs, style, amplitude, y, 0, "x", "y")


def mx_rope_bwd(dy: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, *, style: str = "half",
                amplitude: float = 1.0, dx: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of mx_rope with respect to x: dy turned back.  dx may be dy."""
    dev = dy.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_rope_bwd, locals())
    return _rope(dy, positions, freqs, style, amplitude, dx, 1, "dy", "dx")


def mx_kv_append(k: torch.Tensor, v: torch.Tensor, kv: torch.Tensor, kv_scale: torch.Tensor, page_table: torch.Tensor,
                 kv_lens: torch.Tensor, seq_starts: torch.Tensor, *, freqs: Optional[torch.Tensor] = None,
                 style: str = "half", amplitude: float = 1.0, stream=None) -> None:
    """Keys and values (BF16 [rows][kv_heads][head_dim]) into the cache, at the
    last positions of their sequences; with freqs the keys are turned by their
    positions first (mx_rope).  kv and kv_scale are written in place."""
    dev = k.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_kv_append, locals())
    cache, heads, dim, _ = _cache(kv, kv_scale, page_table, kv_lens, seq_starts, dev)
    shape = (k.shape[0], heads, dim)
    pk, ld_kt, ld_kh = _heads(k, "k", dev, _BF, shape)
    pv, ld_vt, ld_vh = _heads(v, "v", dev, _BF, shape)
    pf, rot = (None, 0) if freqs is None else (_at(freqs, "freqs", dev, _F64, (freqs.numel(),)), 2 * freqs.numel())
    _call("mx_kv_append", dev, cache, pk, ld_kt, ld_kh, pv, ld_vt, ld_vh, shape[0], pf, rot, _style(style), amplitude)


def mx_kv_read(kv: torch.Tensor, kv_scale: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
               seq_starts: torch.Tensor, rows: int, *, k: Optional[torch.Tensor] = None,
               v: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(k, v) [rows][kv_heads][head_dim], BF16 or FP32: the values that the cache
    holds for the rows of seq_starts (kv_lens' sums give whole sequences).  Rows
    behind the last sequence are not written."""
    dev = kv.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_kv_read, locals())
    cache, heads, dim, _ = _cache(kv, kv_scale, page_table, kv_lens, seq_starts, dev)
    given = k if k is not None else v
    dtype = out_dtype if given is None else given.dtype
    if dtype not in _TYPES:
        raise ValueError(f"k and v must be {' or '.join(map(str, _TYPES))}, got {dtype}")
    shape = (rows, heads, dim)
    k, pk = _out_at(k, "k", dev, dtype, *shape)
    v, pv = _out_at(v, "v", dev, dtype, *shape)
    _call("mx_kv_read", dev, cache, rows, pk, pv, _TYPES[dtype])
    return k, v


def mx_kv_attention_workspace_bytes(tokens: int, batch: int, q_heads: int, kv_heads: int, head_dim: int,
                                    max_new: int = 0) -> int:
    """Device scratch mx_kv_attention needs for these sizes, host-only."""
    return _fn("mx_kv_attention_workspace_bytes")(tokens, batch, q_heads, kv_heads, head_dim, max_new)


@functools.lru_cache(maxsize=1024)
def _workspace(device: int, *sizes: int) -> int:
    """mx_kv_attention_workspace_bytes on the current device, which is `device`."""
    return mx_kv_attention_workspace_bytes(*sizes)


def mx_kv_attention(q: torch.Tensor, kv: torch.Tensor, kv_scale: torch.Tensor, page_table: torch.Tensor,
                    kv_lens: torch.Tensor, seq_starts: torch.Tensor, *, scale: Optional[float] = None,
                    causal: bool = True, window: int = 0, max_new: int = 0, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, want_lse: bool = False,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of q (BF16 [rows][q_heads][head_dim]) over the cache: out, or
    (out, lse float32 [rows][q_heads]) with want_lse or lse.

    scale: head_dim^-0.5 if None.  causal: a row sees positions up to its own;
    window > 0: only the last `window` of them.  max_new: the most rows that a
    sequence has in this call (0: not known; a step of few rows then takes more
    launches and up to twice its time, and a single token's weights fewer bits).  Rows behind the last sequence are not written; a row that sees
    nothing gets zeros and -inf.  workspace: device scratch of
    mx_kv_attention_workspace_bytes bytes (a new tensor if None)."""
    dev = q.device
    if stream is not None or dev.index is None or dev.index != _current():
        return _elsewhere(mx_kv_attention, locals())
    cache, kv_heads, dim, batch = _cache(kv, kv_scale, page_table, kv_lens, seq_starts, dev)
    pq, ld_qt, ld_qh = _heads(q, "q", dev, _BF)
    rows, heads, _ = q.shape
    if q.shape[2] != dim:
        raise ValueError(f"q must have heads of {dim}, got {list(q.shape)}")
    if out is None:
        out = torch.empty(rows, heads, dim, dtype=_BF, device=dev)
        po, ld_ot, ld_oh = out.data_ptr(), heads * dim, dim
    else:
        po, ld_ot, ld_oh = _heads(out, "out", dev, _BF, q.shape)
    pl = None
    if lse is not None:
        pl = _at(lse, "lse", dev, torch.float32, (rows, heads))
    elif want_lse:
        lse = torch.empty(rows, heads, dtype=torch.float32, device=dev)
        pl = lse.data_ptr()
    if workspace is None:
        need = _workspace(dev.index, rows, batch, heads, kv_heads, dim, max_new)
        if need:
            workspace = torch.empty(need, dtype=_U8, device=dev)
    pw, nw = _scratch(workspace, dev)
    _call("mx_kv_attention", dev, cache, pq, ld_qt, ld_qh, rows, heads, dim ** -0.5 if scale is None else scale,
          int(causal), window, max_new, po, ld_ot, ld_oh, pl, pw, nw)
    return out if lse is None else (out, lse)
