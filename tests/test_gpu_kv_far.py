"""Offsets beyond 32 bits: rows, pages and heads gigabytes apart give the bytes that
they give side by side."""
import numpy as np
import pytest
import torch

from kv_util import BF, Batch, bf16

pytestmark = pytest.mark.gpu
GIB = 1 << 30


def _apart(t, strides):
    """t's values in a view with those strides of new memory, which holds no more than it must."""
    last = sum((n - 1) * s for n, s in zip(t.shape, strides))
    far = torch.empty(last + 1, dtype=t.dtype, device="cuda").as_strided(t.shape, strides)
    return far.copy_(t)


@pytest.mark.parametrize("dtype,step", [(BF, GIB), (torch.float32, GIB // 2 + 64)])
@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_rope(gpu_lib, style, dtype, step):
    x = torch.randn(4, 3, 96, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    pos = torch.tensor([5, -1, 70000, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    freqs, _ = gpu_lib.mx_rope_frequencies(64)
    want = gpu_lib.mx_rope(x, pos, freqs, style=style)
    for strides in ((step, 96, 1), (96, step, 1)):
        far = _apart(x, strides)
        assert torch.equal(gpu_lib.mx_rope(far, pos, freqs, style=style), want)
        assert gpu_lib.mx_rope(far, pos, freqs, style=style, y=far) is far
        assert torch.equal(far, want)
        del far


@pytest.mark.parametrize("new", [[1, 2, 1], [70, 3, 0]])
@pytest.mark.parametrize("where", ["pages", "heads"])
def test_cache(gpu_lib, where, new):
    heads, q_heads, dim, page = 2, 8, 128, 32
    B = Batch(3, new, [40, 33, 62], heads, dim, page)
    pages, cell = B.kv.shape[1], page * dim
    assert pages >= 6
    if where == "pages":  # keys and values of a page side by side, pages 0.8 GiB apart
        strides = (heads * cell, 13 * GIB // 16, cell, dim, 1)
    else:  # heads 4.5 GiB apart
        strides = (pages * cell, cell, 4 * GIB + GIB // 2, dim, 1)
    far = _apart(B.kv, strides)
    assert far.stride() == strides and max((pages - 1) * strides[1], strides[2]) > 4 * GIB
    far_scale = B.scale.clone()
    k, v, q = (bf16(B.rng, B.rows, h, dim).cuda() for h in (heads, heads, q_heads))
    freqs, _ = gpu_lib.mx_rope_frequencies(dim)
    tables = B.args[2:]
    gpu_lib.mx_kv_append(k, v, *B.args, freqs=freqs)
    gpu_lib.mx_kv_append(_apart(k, (GIB, dim, 1)) if B.rows < 6 else k, v, far, far_scale, *tables, freqs=freqs)
    assert torch.equal(far, B.kv) and torch.equal(far_scale, B.scale)
    for a, b in zip(gpu_lib.mx_kv_read(far, far_scale, *tables, B.rows), gpu_lib.mx_kv_read(*B.args, B.rows)):
        assert torch.equal(a, b)
    for max_new in (0, max(new)):
        want, lse = gpu_lib.mx_kv_attention(q, *B.args, max_new=max_new, want_lse=True)
        got, far_lse = gpu_lib.mx_kv_attention(q, far, far_scale, *tables, max_new=max_new, want_lse=True)
        assert torch.equal(got, want) and torch.equal(far_lse, lse)
        # queries and outputs apart, heads outside the rows
        apart = (dim, 5 * GIB // 16, 1)
        out = _apart(torch.zeros_like(q), apart)
        gpu_lib.mx_kv_attention(_apart(q, apart), far, far_scale, *tables, max_new=max_new, out=out)
        assert torch.equal(out, want)
    assert np.isfinite(want.float().cpu().numpy()).all()
