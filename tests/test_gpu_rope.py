"""Rotary positions and their gradient against the 64-bit form (tests/kv_ref.py).

Tolerances.  cos and sin are within 2^-40 of the angle's (64-bit angle and
series) and rounded to FP32 after the amplitude: 2 half steps of 2^-24; the two
products and their sum round three times more at most, each relative to a term or
to the result, which the terms bound: 5 * 2^-24 * amplitude * (|x0| + |x1|), and 2^-40
of it for the angle.  The BF16 result adds its rounding, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import kv_ref as ref

pytestmark = pytest.mark.gpu


def _freqs(rot, base=1e4):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


def _near(got, want, mag, dtype):
    tol = (5 * 2.0 ** -24 + 2.0 ** -39) * mag + (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24) * np.abs(want) + 1e-38
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err / tol).max()


def _mag(x, rot, style, amplitude):
    """amplitude * (|x0| + |x1|) of every element's pair; 0 for copied ones."""
    a, m = np.abs(x), np.zeros_like(x)
    n = rot // 2
    if style == "half":
        m[..., :n] = m[..., n:rot] = a[..., :n] + a[..., n:rot]
    else:
        m[..., 0:rot:2] = m[..., 1:rot:2] = a[..., 0:rot:2] + a[..., 1:rot:2]
    return m * abs(amplitude)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("T,H,D,rot,amp", [(1, 1, 16, 16, 1.0), (3, 5, 80, 32, 1.25), (17, 32, 128, 128, 1.0), (2, 7, 24, 16, 1.0),
                                           (33, 3, 64, 48, 0.5), (5, 2, 512, 512, 1.0), (4, 1, 512, 16, -1.0), (9, 11, 104, 96, 1.0),
                                           (4100, 2, 64, 64, 1.0), (4099, 1, 72, 32, 1.5)])
def test_rope_and_gradient(gpu_lib, T, H, D, rot, amp, style, dtype):
    g = torch.Generator().manual_seed(T * D + rot)
    x = torch.randn(T, H, D, generator=g).to(dtype)
    pos = torch.randint(-5, 200000, (T,), generator=g).int()
    pos[0] = 0
    f = _freqs(rot, 1e6)
    fd, pd = torch.from_numpy(f).cuda(), pos.cuda()
    y = gpu_lib.mx_rope(x.cuda(), pd, fd, style=style, amplitude=amp)
    dx = gpu_lib.mx_rope_bwd(x.cuda(), pd, fd, style=style, amplitude=amp)
    xn = x.double().numpy()
    mag = _mag(xn, rot, style, amp)
    _near(y, ref.rope(xn, pos.numpy(), f, style, amp), mag, dtype)
    _near(dx, ref.rope(xn, pos.numpy(), f, style, amp, inverse=True), mag, dtype)
    assert torch.equal(y[..., rot:].cpu(), x[..., rot:]) and torch.equal(dx[..., rot:].cpu(), x[..., rot:])
    if amp == 1.0:
        assert torch.equal(y[0].cpu(), x[0])  # position 0


def test_far_positions_lose_nothing(gpu_lib):
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 1 << 24, (1 << 24) + 1], dtype=torch.int32)
    f = _freqs(64)
    x = torch.randn(5, 2, 64, generator=torch.Generator().manual_seed(1))
    y = gpu_lib.mx_rope(x.cuda(), pos.cuda(), torch.from_numpy(f).cuda())
    # the reference's angle is rounded to 2^-53 of up to 2^31, ours too: 2^-21 either way
    want = ref.rope(x.double().numpy(), pos.numpy(), f)
    tol = (5 * 2.0 ** -24 + 2 * 2.0 ** -21) * _mag(x.double().numpy(), 64, "half", 1.0)
    assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()


def test_gradient_is_that_of_differences(gpu_lib):
    """The rotation is linear: (f(x + h) - f(x)) / h . dy = h-direction . dx."""
    g = torch.Generator().manual_seed(7)
    x, h, dy = (torch.randn(6, 3, 96, generator=g) for _ in range(3))
    pos = torch.randint(0, 5000, (6,), generator=g).int().cuda()
    f = torch.from_numpy(_freqs(64)).cuda()
    for style in ("half", "interleaved"):
        kw = dict(style=style, amplitude=1.5)
        up = gpu_lib.mx_rope((x + h).cuda(), pos, f, **kw).double() - gpu_lib.mx_rope(x.cuda(), pos, f, **kw).double()
        lhs = (up.cpu() * dy.double()).sum()
        rhs = (h.double() * gpu_lib.mx_rope_bwd(dy.cuda(), pos, f, **kw).double().cpu()).sum()
        # every value is off by less than 8 * 2^-24 * 1.5 * its pair's magnitude (x + h is rounded too)
        bound = 8 * 2.0 ** -24 * 1.5 * 2 * float(((x.abs() + h.abs() + (x + h).abs()).double().sum(-1) * dy.abs().double().sum(-1)).sum())
        assert abs(float(lhs - rhs)) <= bound


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_strides_and_in_place(gpu_lib, style, dtype):
    g = torch.Generator().manual_seed(11)
    T, H, D = 13, 4, 64
    base = torch.randn(T, H + 6, D + 16, generator=g).to(dtype).cuda()
    pos = torch.randint(0, 999, (T,), generator=g).int().cuda()
    f = torch.from_numpy(_freqs(32)).cuda()
    view = base[:, 2:2 + H, :D]
    want = gpu_lib.mx_rope(view.contiguous(), pos, f, style=style)
    assert torch.equal(gpu_lib.mx_rope(view, pos, f, style=style), want)
    # heads outside the rows
    turned = view.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.zeros_like(turned)
    assert turned.stride(0) == D and gpu_lib.mx_rope(turned, pos, f, style=style, y=out) is out
    assert torch.equal(out, want)
    # in place, the rest of the buffer untouched
    before = base.clone()
    gpu_lib.mx_rope(view, pos, f, style=style, y=view)
    assert torch.equal(view, want)
    base[:, 2:2 + H, :D] = before[:, 2:2 + H, :D]
    assert torch.equal(base, before)
    gpu_lib.mx_rope_bwd(view, pos, f, style=style, dx=view)
    assert torch.equal(view, gpu_lib.mx_rope_bwd(before[:, 2:2 + H, :D], pos, f, style=style))


def test_special_values_stay_in_their_pair(gpu_lib):
    x = torch.ones(2, 2, 64)
    x[0, 0, 3], x[1, 1, 40], x[0, 1, 63] = float("nan"), float("inf"), float("nan")
    y = gpu_lib.mx_rope(x.cuda(), torch.tensor([1, 2], dtype=torch.int32).cuda(), torch.from_numpy(_freqs(32)).cuda()).cpu()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 0, 3] = want[0, 0, 19] = want[0, 1, 63] = want[1, 1, 40] = True
    assert torch.equal(bad, want)


def test_empty_calls_and_binding_refusals(gpu_lib):
    f = torch.from_numpy(_freqs(32)).cuda()
    pos = torch.zeros(0, dtype=torch.int32).cuda()
    assert gpu_lib.mx_rope(torch.zeros(0, 3, 64).cuda(), pos, f).shape == (0, 3, 64)
    assert gpu_lib.mx_rope(torch.zeros(2, 0, 64).cuda(), torch.zeros(2, dtype=torch.int32).cuda(), f).shape == (2, 0, 64)
    x = torch.zeros(4, 2, 64).cuda()
    p4 = torch.zeros(4, dtype=torch.int32).cuda()
    for bad in (dict(x=x.half()), dict(positions=p4.long()), dict(positions=p4[:3]), dict(freqs=f.float()), dict(style="quarter"),
                dict(x=x[0]), dict(x=x.transpose(1, 2)), dict(y=torch.zeros(4, 2, 32).cuda()), dict(y=x.bfloat16()),
                dict(positions=p4.cpu())):
        with pytest.raises(ValueError):
            gpu_lib.mx_rope(**dict(dict(x=x, positions=p4, freqs=f), **bad))
    for bad in (dict(x=x[:, :1].expand(4, 2, 64)), dict(freqs=f[:7].contiguous()), dict(y=x[:, :, :].flip(0)[:4].as_strided((4, 2, 64), (128, 32, 1)))):
        with pytest.raises(gpu_lib.MxError):
            gpu_lib.mx_rope(**dict(dict(x=x, positions=p4, freqs=f), **bad))
