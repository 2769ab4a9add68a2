"""CPU checks of the ABI's third part (include/mxfp8_kv.h): every declared
entry point is exported and bound, the rotary frequencies agree with their
formulas, and invalid arguments are refused before HIP is touched (fake
pointers are never dereferenced)."""
import ctypes
import inspect
import math
import os
import re

import numpy as np
import pytest
import torch

import kv_ref as ref
import mxfp8_block_scaled_08_amd as mx
from mxfp8_block_scaled_08_amd import kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D, E, F, G, H, I, J = (i << 40 for i in range(1, 11))
BF, F32 = mx.MX_BF16, mx.MX_F32
INV, SHAPE, ALIGN, OVER, UNSUP = (mx.MX_ERR_INVALID_ARG, mx.MX_ERR_SHAPE, mx.MX_ERR_ALIGN, mx.MX_ERR_OVERLAP,
                                  mx.MX_ERR_UNSUPPORTED)


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxfp8_kv.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mx_[a-z_0-9]+)\s*\(", text)))
    assert len(names) == 6
    raw = ctypes.CDLL(mx.lib_path())
    for n in names:
        assert hasattr(raw, n) and hasattr(mx, n) and n in mx.__all__, n
        decl = re.search(n + r"\s*\((.*?)\)\s*;", text, flags=re.S).group(1)
        assert len(kv._ARGS[n]) == decl.count(",") + 1, n
        if not n.endswith(("_bytes", "_frequencies")):
            assert "stream" in inspect.signature(getattr(mx, n)).parameters, n
    assert "stream" in inspect.signature(mx.mx_rope_bwd).parameters
    fields = re.search(r"typedef struct mx_kv_cache \{(.*?)\}", text, flags=re.S).group(1)
    want = re.findall(r"(\w+)\s*[,;]", fields)
    assert [f for f, _ in kv._Cache._fields_] == want
    assert ctypes.sizeof(kv._Cache) == 8 * len(want)


# rotary frequencies: 64-bit formulas; a power of a quotient loses a few ulp


@pytest.mark.parametrize("rot", [2, 16, 64, 128, 256])
@pytest.mark.parametrize("base", [1e4, 1e6])
def test_frequencies(rot, base):
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    near = dict(rtol=1e-13, atol=0)
    got, amp = mx.mx_rope_frequencies(rot, base, device="cpu")
    assert got.dtype == torch.float64 and amp == 1.0
    np.testing.assert_allclose(got.numpy(), f, **near)
    got, amp = mx.mx_rope_frequencies(rot, base, "linear", 8.0, device="cpu")
    np.testing.assert_allclose(got.numpy(), f / 8, **near)
    if rot > 2:
        got, amp = mx.mx_rope_frequencies(rot, base, "ntk", 4.0, device="cpu")
        assert amp == 1.0
        np.testing.assert_allclose(got.numpy()[0], 1.0, **near)
        np.testing.assert_allclose(got.numpy()[-1], f[-1] / 4, **near)
        np.testing.assert_allclose(got.numpy(), (base * 4.0 ** (rot / (rot - 2))) ** (-2.0 * i / rot), **near)
    got, amp = mx.mx_rope_frequencies(rot, base, "yarn", 4.0, 32768, device="cpu")
    turns = 32768 * f / (2 * math.pi)
    keep = np.clip((turns - 1) / 31, 0, 1)
    np.testing.assert_allclose(got.numpy(), f * keep + f / 4 * (1 - keep), **near)
    assert (got.numpy()[turns > 32] == f[turns > 32]).all() or np.allclose(got.numpy()[turns > 32], f[turns > 32], **near)
    assert amp == np.float32(1 + 0.1 * math.log(4.0))
    same, amp = mx.mx_rope_frequencies(rot, base, "yarn", 1.0, 32768, device="cpu")
    np.testing.assert_allclose(same.numpy(), f, **near)
    assert amp == 1.0


def test_frequencies_refusals():
    buf = (ctypes.c_double * 64)()
    amp = ctypes.c_float()
    f = lambda *a: kv._fn("mx_rope_frequencies")(*a, ctypes.addressof(buf), ctypes.addressof(amp))  # noqa: E731
    assert f(64, 1e4, 0, 1.0, 0) == mx.MX_OK
    for bad in ((63, 1e4, 0, 1.0, 0), (0, 1e4, 0, 1.0, 0), (2, 1e4, 2, 2.0, 0), (64, 0.0, 0, 1.0, 0), (64, math.inf, 0, 1.0, 0),
                (64, 1e4, 4, 1.0, 0), (64, 1e4, -1, 1.0, 0), (64, 1e4, 1, 0.5, 0), (64, 1e4, 1, math.nan, 0),
                (64, 1e4, 3, 2.0, 0)):
        assert f(*bad) == INV, bad
        assert "mx_rope_frequencies" in mx.mx_last_error()
    assert kv._fn("mx_rope_frequencies")(64, 1e4, 0, 1.0, 0, None, ctypes.addressof(amp)) == INV
    with pytest.raises(ValueError, match="scaling"):
        mx.mx_rope_frequencies(64, scaling="cubic", device="cpu")
    with pytest.raises(mx.MxError):
        mx.mx_rope_frequencies(64, base=-1.0, device="cpu")


ROPE = dict(x=A, dtype=BF, tokens=4, heads=3, dim=64, ld_xt=192, ld_xh=64, pos=B, freqs=C, rot=64, style=0, amp=1.0, inv=0,
            y=D, ld_yt=192, ld_yh=64)


def test_rope_refusals():
    def r(status, word="", **kw):
        args = dict(ROPE, **kw)
        assert len(args) == len(ROPE)
        assert kv._fn("mx_rope")(*args.values(), None) == status, mx.mx_last_error()
        assert "mx_rope" in mx.mx_last_error() and word in mx.mx_last_error()

    r(INV, "dtype", dtype=2)
    r(INV, tokens=-1)
    r(INV, heads=-1)
    r(INV, dim=0)
    r(SHAPE, "head_dim", dim=68)
    r(SHAPE, "rot_dim", rot=0)
    r(SHAPE, "rot_dim", rot=24)
    r(SHAPE, "rot_dim", rot=80)
    r(INV, "style", style=2)
    r(INV, "amplitude", amp=math.nan)
    r(UNSUP, dim=520, ld_xh=520, ld_yh=520, ld_xt=2000, ld_yt=2000)
    r(UNSUP, tokens=1 << 24)
    r(UNSUP, ld_xt=1 << 40)
    r(UNSUP, ld_yh=-64)
    r(INV, "overlap", ld_xh=56)
    r(INV, "overlap", ld_yt=128)
    r(INV, "overlap", ld_yt=0)
    r(INV, "null", x=None)
    r(INV, "null", y=None)
    r(INV, "null", pos=None)
    r(INV, "null", freqs=None)
    r(ALIGN, x=A + 8)
    r(ALIGN, y=D + 2)
    r(ALIGN, ld_xt=196)
    r(ALIGN, ld_xh=66, ld_xt=264)
    r(ALIGN, pos=B + 2)
    r(ALIGN, freqs=C + 4)
    r(ALIGN, x=A + 8, dtype=F32)
    r(OVER, y=A + 16)
    r(OVER, y=A, ld_yt=256)
    r(OVER, y=B - 16)
    r(OVER, y=C)
    for ok in (dict(tokens=0), dict(heads=0)):
        assert kv._fn("mx_rope")(*dict(ROPE, **ok).values(), None) == mx.MX_OK


CACHE = dict(k=A, v=B, k_scale=C, v_scale=D, num_pages=10, kv_heads=2, page_size=64, head_dim=128, ld_page=2 * 64 * 128,
             ld_head=64 * 128, ld_token=128, page_table=E, max_pages=4, kv_lens=F, seq_starts=G, batch=3)


def _cache(**kw):
    return ctypes.byref(kv._Cache(**dict(CACHE, **kw)))


APPEND = dict(k=H, ld_kt=512, ld_kh=128, v=H + 512, ld_vt=512, ld_vh=128, tokens=5, freqs=I, rot=128, style=0, amp=1.0)
READ = dict(tokens=5, k=H, v=I, dtype=BF)
ATTENTION = dict(q=H, ld_qt=1024, ld_qh=128, tokens=5, q_heads=8, scale=0.1, causal=1, window=0, max_new=0, out=I, ld_ot=1024,
                 ld_oh=128, lse=J, ws=J << 1, ws_bytes=1 << 40)
CALLS = [("mx_kv_append", APPEND), ("mx_kv_read", READ), ("mx_kv_attention", ATTENTION)]


@pytest.mark.parametrize("name,base", CALLS)
def test_cache_refusals(name, base):
    def r(status, word="", **kw):
        got = kv._fn(name)(_cache(**kw), *base.values(), None)
        assert got == status, mx.mx_last_error()
        assert name in mx.mx_last_error() and word in mx.mx_last_error()

    assert kv._fn(name)(None, *base.values(), None) == INV
    r(INV, num_pages=0)
    r(INV, kv_heads=0)
    r(INV, max_pages=0)
    r(INV, batch=-1)
    r(INV, page_size=0)
    r(UNSUP, "head_dim", head_dim=96)
    r(UNSUP, "head_dim", head_dim=256)
    r(UNSUP, "page_size", page_size=48)
    r(UNSUP, "page_size", page_size=8)
    r(UNSUP, "page_size", page_size=2048)
    r(UNSUP, num_pages=1 << 30)
    r(UNSUP, max_pages=1 << 24)
    r(UNSUP, kv_heads=2048, ld_head=128)
    r(UNSUP, batch=65537)
    r(UNSUP, "ld_token", ld_token=1 << 20)
    r(UNSUP, ld_token=-128)
    r(INV, "overlap", ld_token=64)
    r(INV, "overlap", ld_head=1024)
    r(INV, "overlap", ld_page=128)
    r(INV, "overlap", ld_page=0)
    r(ALIGN, k=A + 8)
    r(ALIGN, ld_token=136, ld_head=1 << 20, ld_page=1 << 22)
    r(ALIGN, page_table=E + 2)
    r(ALIGN, kv_lens=F + 1)
    r(ALIGN, seq_starts=G + 4)
    for p in ("k", "v", "k_scale", "v_scale", "page_table", "kv_lens", "seq_starts"):
        r(INV, "null", **{p: None})
    assert kv._fn(name)(_cache(batch=0), *base.values(), None) == mx.MX_OK
    assert kv._fn(name)(_cache(), *dict(base, tokens=0).values(), None) == mx.MX_OK
    assert kv._fn(name)(_cache(), *dict(base, tokens=-1).values(), None) == INV
    assert kv._fn(name)(_cache(), *dict(base, tokens=1 << 28).values(), None) == UNSUP


def _refused(name, base, status, word="", cache=None, **kw):
    args = dict(base, **kw)
    assert len(args) == len(base)
    assert kv._fn(name)(_cache(**(cache or {})), *args.values(), None) == status, mx.mx_last_error()
    assert name in mx.mx_last_error() and word in mx.mx_last_error()


def test_append_refusals():
    r = lambda st, word="", cache=None, **kw: _refused("mx_kv_append", APPEND, st, word, cache, **kw)  # noqa: E731
    r(SHAPE, "rot_dim", rot=136)
    r(SHAPE, "rot_dim", rot=8)
    r(INV, "style", style=3)
    r(INV, "amplitude", amp=math.inf)
    r(INV, "null", k=None)
    r(INV, "null", v=None)
    r(ALIGN, k=H + 2)
    r(ALIGN, ld_vt=516)
    r(ALIGN, freqs=I + 4)
    r(INV, "overlap", ld_kt=128)
    r(OVER, k=A + 4096)
    r(OVER, v=C)
    r(OVER, freqs=D + 8)
    r(OVER, cache=dict(v=A + 128))
    r(OVER, cache=dict(k_scale=A))
    r(OVER, cache=dict(page_table=D + 4))
    r(OVER, cache=dict(v_scale=C + 16))
    # keys and values that alternate, but too near
    r(OVER, cache=dict(v=A + 64 * 128, ld_page=3 * 64 * 128))


def test_read_refusals():
    r = lambda st, word="", cache=None, **kw: _refused("mx_kv_read", READ, st, word, cache, **kw)  # noqa: E731
    r(INV, "dtype", dtype=3)
    r(ALIGN, k=H + 8)
    r(ALIGN, v=I + 2)
    r(OVER, k=A)
    r(OVER, v=H + 64)
    r(OVER, v=E)
    assert kv._fn("mx_kv_read")(_cache(), 5, None, None, BF, None) == mx.MX_OK


def test_attention_refusals():
    r = lambda st, word="", cache=None, **kw: _refused("mx_kv_attention", ATTENTION, st, word, cache, **kw)  # noqa: E731
    r(INV, "q_heads", q_heads=7)
    r(INV, "q_heads", q_heads=1)
    r(INV, "scale", scale=-0.1)
    r(INV, "scale", scale=math.nan)
    r(INV, "window", window=-1)
    r(INV, "window", window=5, causal=0)
    r(INV, "max_new", max_new=-1)
    r(UNSUP, "1024", q_heads=4096, ld_qt=4096 * 128, ld_ot=4096 * 128)
    r(UNSUP, tokens=1 << 26)
    r(INV, "null", q=None)
    r(INV, "null", out=None)
    r(ALIGN, q=H + 8)
    r(ALIGN, out=I + 8)
    r(ALIGN, lse=J + 2)
    r(INV, "overlap", ld_ot=512)
    r(OVER, out=H)
    r(OVER, out=A)
    r(OVER, lse=I + 8)
    r(OVER, lse=G)
    r(INV, "workspace", ws=None)
    r(INV, "workspace", ws_bytes=16)
    r(INV, "workspace", ws_bytes=-1)
    r(ALIGN, ws=(J << 1) + 8)
    r(OVER, "workspace", ws=H)
    r(OVER, "workspace", ws=I)
    r(OVER, "workspace", ws=B)


def test_workspace_query():
    f = mx.mx_kv_attention_workspace_bytes
    assert f(64, 64, 32, 8, 128, 1) > 0
    assert f(0, 64, 32, 8, 128) == f(64, 0, 32, 8, 128) == f(64, 64, 4, 8, 128) == f(1 << 27, 1, 1, 1, 128) == 0
    assert f(64, 64, 32, 8, 128, -1) == 0
    # never more than a fraction of the card
    assert f(20480, 64, 32, 8, 128) < 1 << 30 and f(128, 1, 1024, 1, 128) < 1 << 30


def test_binding_refuses_on_the_host():
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pos, freqs = torch.zeros(4, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="device tensor"):
        mx.mx_rope(t, pos, freqs)
    with pytest.raises(ValueError, match="device tensor"):
        mx.mx_rope_bwd(t, pos, freqs)
    cache = (torch.zeros(2, 3, 2, 16, 64, dtype=torch.uint8), torch.zeros(2, 3, 2, 1, dtype=torch.uint8),
             torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="device tensor"):
        mx.mx_kv_append(t, t, *cache)
    with pytest.raises(ValueError, match="device tensor"):
        mx.mx_kv_read(*cache, 4)
    with pytest.raises(ValueError, match="device tensor"):
        mx.mx_kv_attention(t, *cache)


# the reference itself, against the definitions spelled out


def test_reference_encoding_is_the_nearest_code():
    rng = np.random.default_rng(3)
    v = np.concatenate([rng.standard_normal(2000) * 100, ref.E4M3[:127], -ref.E4M3[:127], (ref.E4M3[:126] + ref.E4M3[1:127]) / 2,
                        rng.standard_normal(500) * 1e-3, [448.0, -448.0, 0.0, -0.0]])
    v = np.clip(v, -448, 448)
    for code in (127, 100, 140):
        q, bad = ref.encode(v * 2.0 ** (code - 127), code)
        assert not bad.any()
        order = np.r_[0:127, 128:255]  # codes without NaN
        gap = np.abs(ref.E4M3[order][None] - v[:, None])
        best = gap.min(1)
        got = np.abs(ref.E4M3[q] - v)
        assert (got == best).all()
        tie = (gap == best[:, None]).sum(1) > 1
        assert ((q[tie] & 1) == 0).all()  # (both zeros are even)
        assert (np.signbit(ref.E4M3[q]) == np.signbit(v)).all()


def test_reference_scale_keeps_a_block_within_448():
    for a in (448.0, 449.0, 447.9, 1.0, 1.75, 1.7500001, 3e38, 1e-30, 2.0 ** -133):
        c = ref.scale_code(a)
        assert a <= 448 * 2.0 ** (c - 127) and (c == 0 or a > 448 * 2.0 ** (c - 128)), a
    assert ref.scale_code(0.0) == 0


def test_reference_rotation_is_a_complex_product():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((5, 2, 48))
    pos, f = np.array([0, 1, 7, -3, 100000]), 10.0 ** -np.arange(16.0)
    z = np.exp(1j * pos[:, None, None] * f) * float(np.float32(1.5))
    half = (x[..., :16] + 1j * x[..., 16:32]) * z
    np.testing.assert_allclose(ref.rope(x, pos, f, "half", 1.5)[..., :32], np.concatenate([half.real, half.imag], -1), atol=1e-12)
    inter = (x[..., 0:32:2] + 1j * x[..., 1:32:2]) * z
    got = ref.rope(x, pos, f, "interleaved", 1.5)
    np.testing.assert_allclose(got[..., 0:32:2], inter.real, atol=1e-12)
    np.testing.assert_allclose(got[..., 1:32:2], inter.imag, atol=1e-12)
    assert (got[..., 32:] == x[..., 32:]).all()
    np.testing.assert_allclose(ref.rope(ref.rope(x, pos, f), pos, f, inverse=True), x, atol=1e-12)


@pytest.mark.parametrize("name,base", CALLS)
def test_limits_of_the_cache(name, base):
    """The last sizes that are taken and the first that are refused, where 32-bit offsets would wrap."""
    def r(status, **kw):
        none = dict(base, tokens=0, **({"q_heads": 4 * kw.get("kv_heads", 2)} if "q_heads" in base else {}))
        assert kv._fn(name)(_cache(**kw), *none.values(), None) == status, mx.mx_last_error()

    r(UNSUP, ld_page=1 << 32)
    r(mx.MX_OK, ld_page=(1 << 32) - 16)
    r(mx.MX_OK, num_pages=1, ld_page=1 << 50)  # a stride over one page is not looked at
    r(UNSUP, kv_heads=1, ld_page=64 * 128, page_size=64, num_pages=1 << 29)  # 2^31 blocks
    r(mx.MX_OK, kv_heads=1, ld_page=64 * 128, page_size=64, num_pages=(1 << 29) - 1)
    r(UNSUP, kv_heads=1024, num_pages=1, ld_head=1 << 36)
    r(mx.MX_OK, kv_heads=1024, num_pages=1, ld_head=(1 << 36) - 16)
    r(UNSUP, batch=1 << 16, kv_heads=128, ld_head=64 * 128, ld_page=1 << 20)
    r(mx.MX_OK, batch=1 << 16, kv_heads=127, ld_head=64 * 128, ld_page=1 << 20)
    r(UNSUP, max_pages=1 << 20, page_size=1024, ld_head=1 << 17, ld_page=1 << 18)
    r(mx.MX_OK, max_pages=(1 << 20) - 1, page_size=1024, ld_head=1 << 17, ld_page=1 << 18)
    # pages outside or inside the heads, slots outside both
    r(mx.MX_OK, ld_page=64 * 128, ld_head=10 * 64 * 128)
    r(mx.MX_OK, ld_page=128, ld_head=1280, ld_token=2560)
    r(INV, ld_page=128, ld_head=1280, ld_token=2432)


def test_workspace_query_and_call_take_the_same_sizes():
    """Both sides of each limit: the query is above 0 just where the call takes the sizes (asked of a call without a
    workspace, which says so last)."""
    def take(tokens, batch, q_heads, kv_heads, dim, max_new=0):
        need = mx.mx_kv_attention_workspace_bytes(tokens, batch, q_heads, kv_heads, dim, max_new)
        c = _cache(kv_heads=kv_heads, head_dim=dim, batch=batch, num_pages=2, page_size=16, ld_token=128, ld_head=16 * 128,
                   ld_page=1 << 22)
        args = dict(ATTENTION, tokens=tokens, q_heads=q_heads, max_new=max_new, ws=None, ws_bytes=0, lse=None, q=1 << 51,
                    out=1 << 52, ld_qt=q_heads * 128, ld_ot=q_heads * 128)
        st = kv._fn("mx_kv_attention")(c, *args.values(), None)
        if need:
            assert st == INV and "workspace" in mx.mx_last_error(), (st, mx.mx_last_error())
        else:
            assert st in (INV, UNSUP) and "workspace" not in mx.mx_last_error(), (st, mx.mx_last_error())
        return need > 0

    assert take(5, 3, 8, 2, 128) and take(5, 3, 8, 2, 64) and take(5, 3, 2, 2, 64, 1)
    assert not take(5, 3, 7, 2, 128) and not take(5, 3, 1, 2, 128) and not take(5, 3, 8, 2, 128, -1)
    for dim in (32, 96, 192, 256, 1 << 40, 1 << 62):
        assert not take(5, 3, 8, 2, dim)
    assert take(5, 3, 1024, 1024, 64) and not take(5, 3, 1025, 1025, 64) and not take(5, 3, 2048, 2048, 64)
    assert take(5, 3, 1024, 1, 64) and not take(5, 3, 1025, 1, 64) and take(5, 3, 2048, 2, 64) and not take(5, 3, 2050, 2, 64)
    assert take(5, 65536, 127, 127, 64) and not take(5, 65536, 128, 128, 64) and not take(5, 65537, 1, 1, 64)
    assert not take(-1, 3, 8, 2, 128) and not take(5, -1, 8, 2, 128) and not take(5, 3, 8, 0, 128) and not take(5, 3, 8, -2, 128)
    # tokens * q_heads below 2^27, the whole quotient's remainder too
    for heads in (1, 3, 5, 8, 1000):
        last = ((1 << 27) - 1) // heads
        assert take(last, 3, heads, 1, 64) and not take(last + 1, 3, heads, 1, 64), heads
    assert take((1 << 27) - 1, 1, 1, 1, 128) and not take(1 << 27, 1, 1, 1, 128) and not take(1 << 62, 1, 1, 1, 128)
    assert not take(5, 3, 1 << 62, 2, 128)


def test_yarn_over_the_pairs():
    """The ramp over the pairs' numbers.  Base 10^6, 128 elements, 32768 positions: pair 23.6 turns 32 times, pair 39.7 once
    (64 ln(32768 / (64 pi)) / ln 10^6 and 64 ln(32768 / (2 pi)) / ln 10^6), so pairs up to 23 are kept, from 40 on
    interpolated, pair 31 keeps 9 parts of 17."""
    near = dict(rtol=1e-13, atol=0)
    f = 1e6 ** (-2.0 * np.arange(64) / 128)
    got, amp = mx.mx_rope_frequencies(128, 1e6, "yarn_pairs", 4.0, 32768, device="cpu")
    got = got.numpy()
    assert amp == np.float32(1 + 0.1 * math.log(4.0))
    np.testing.assert_allclose(got[:24], f[:24], **near)
    np.testing.assert_allclose(got[40:], f[40:] / 4, **near)
    keep = (40 - np.arange(24, 40)) / 17
    assert keep[31 - 24] == 9 / 17
    np.testing.assert_allclose(got[24:40], f[24:40] * keep + f[24:40] / 4 * (1 - keep), **near)
    # the paper's ramp over the turns keeps less of it
    other, _ = mx.mx_rope_frequencies(128, 1e6, "yarn", 4.0, 32768, device="cpu")
    assert other.numpy()[31] < 0.65 * got[31]
    # nothing to scale; all pairs fast; all pairs slow but the first; a ramp that starts before the first pair
    np.testing.assert_allclose(mx.mx_rope_frequencies(128, 1e6, "yarn_pairs", 1.0, 32768, device="cpu")[0].numpy(), f, **near)
    np.testing.assert_allclose(mx.mx_rope_frequencies(128, 1e6, "yarn_pairs", 4.0, 1 << 40, device="cpu")[0].numpy(), f, **near)
    got = mx.mx_rope_frequencies(128, 1e6, "yarn_pairs", 4.0, 1, device="cpu")[0].numpy()
    np.testing.assert_allclose(got[1:], f[1:] / 4, **near)
    # 64 ln(64 / (2 pi)) / ln 10^6 = 10.75: from pair 11 on interpolated, the ramp from pair 0
    got = mx.mx_rope_frequencies(128, 1e6, "yarn_pairs", 8.0, 64, device="cpu")[0].numpy()
    keep = np.clip((11 - np.arange(64)) / 11, 0, 1)
    np.testing.assert_allclose(got, f * keep + f / 8 * (1 - keep), **near)
    assert mx.mx_rope_frequencies(2, 1e4, "yarn_pairs", 4.0, 4096, device="cpu")[0].shape == (1,)


def test_yarn_over_the_pairs_refusals():
    buf = (ctypes.c_double * 64)()
    amp = ctypes.c_float()
    f = lambda *a: kv._fn("mx_rope_frequencies")(*a, ctypes.addressof(buf), ctypes.addressof(amp))  # noqa: E731
    assert f(64, 1e4, mx.MX_ROPE_YARN_PAIRS, 4.0, 4096) == mx.MX_OK
    for bad in ((64, 1.0, 4, 4.0, 4096), (64, 0.5, 4, 4.0, 4096), (64, 1e4, 4, 4.0, 0), (64, 1e4, 4, 0.9, 4096), (63, 1e4, 4, 4.0, 4096),
                (64, 1e4, 5, 4.0, 4096)):
        assert f(*bad) == INV, bad
        assert "mx_rope_frequencies" in mx.mx_last_error()
