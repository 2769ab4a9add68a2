"""Routing of tokens to experts, its gradient and the combine's gradient
against the 64-bit reference (tests/fp4_ref.py).

Ids are whole numbers and must be equal.  Tolerances: a weight is a chain of
an exponential (2 ulp), a sum and a division in FP32 after x - max was rounded
once, so its relative error is at most (|x - max| + 64) * 2^-24; a gradient is
such a weight times differences of the incoming gradients, at most
scale * s * (|g_j| + |D|), with the same factor; a BF16 result adds 2^-8.
"""
import numpy as np
import pytest
import torch

import fp4_ref as ref
import mxsynth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _logits(rng, T, E, dtype, spread=4.0):
    x = torch.from_numpy((rng.standard_normal((T, E)) * spread).astype(np.float32))
    return x.to(dtype)


def _check(mx, x, topk, score, **kw):
    kw = dict(kw)
    bias, mask = kw.pop("bias", None), kw.pop("mask", None)
    groups, keep, gtop = kw.pop("num_groups", 1), kw.pop("topk_groups", 1), kw.pop("group_top", 1)
    renorm, scale = kw.pop("renormalize", True), kw.pop("scale", 1.0)
    ids, w = mx.mx_moe_route(x.cuda(), topk, score=score, bias=None if bias is None else torch.from_numpy(bias).cuda(),
                             num_groups=groups, topk_groups=keep, group_top=gtop, renormalize=renorm, scale=scale,
                             mask=None if mask is None else torch.from_numpy(mask).cuda())
    torch.cuda.synchronize()
    xn = x.float().numpy()
    rid, rw = ref.route(xn, topk, score == "softmax", bias, groups, keep, gtop, renorm, scale, mask)
    got = ids.cpu().numpy()
    assert np.array_equal(got, rid), f"{(got != rid).any(1).sum()} rows differ, first {np.argwhere(got != rid)[:3]}"
    fin = np.where(np.isfinite(xn), xn, 0)
    span = np.abs(fin).max() * 2
    err = np.abs(w.cpu().numpy() - rw)
    assert (err <= (span + 64) * U * rw + 1e-44).all(), (err / np.maximum(rw, 1e-300)).max()
    return ids, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (7, 64, 1), (33, 65, 8), (130, 128, 8), (61, 160, 6),
                                   (29, 256, 17), (18, 513, 32), (9, 1024, 8), (40, 500, 8), (21, 1000, 4), (50, 100, 3),
                                   (13, 260, 9)])
def test_route_and_gradient(gpu_lib, T, E, k, renorm, score):
    rng = np.random.default_rng(T * E + k)
    for dtype in (torch.float32, torch.bfloat16):
        x = _logits(rng, T, E, dtype)
        ids, w = _check(gpu_lib, x, k, score, renormalize=renorm, scale=1.5)
        g = rng.standard_normal((T, k)).astype(np.float32)
        dx = gpu_lib.mx_moe_route_bwd(torch.from_numpy(g).cuda(), x.cuda(), ids, score=score, renormalize=renorm,
                                      scale=1.5)
        xn = x.float().numpy()
        want = ref.route_bwd(xn, ids.cpu().numpy(), g, score == "softmax", renorm, 1.5)
        # the size of what is added up at each expert: its score times the gradients
        size = np.abs(want) + _sizes(xn, ids.cpu().numpy(), g, score == "softmax", renorm) * 1.5
        tol = (np.abs(xn).max() * 2 + 64 + k) * 2 * U * size + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
        # the 64-bit reference's own rounding: with renormalized softmax the sum of ds_k s_k is
        # zero, of terms up to 2 * 1.5 * max |g|, and leaves k * 2^-53 of them at every expert
        tol = tol + k * 2.0 ** -50 * np.abs(g).max() + 1e-38
        err = np.abs(dx.float().cpu().numpy() - want)
        assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(4301, 128, 8), (4500, 70, 20), (2301, 256, 8), (2100, 131, 32), (2303, 512, 8),
                                   (2150, 300, 17)])
def test_many_tokens(gpu_lib, T, E, k, score):
    """More tokens than eight waves a compute unit of the wide form: half the lanes a token."""
    if torch.cuda.get_device_properties(0).multi_processor_count > 256:
        pytest.skip("sized for 256 compute units")
    test_route_and_gradient(gpu_lib, T, E, k, score == "softmax", score)
    rng = np.random.default_rng(T)
    G = {128: 8, 70: 7, 256: 8, 131: 1, 512: 16, 300: 10}[E]
    keep = max(1, (G + 1) // 2)
    bias = rng.standard_normal(E).astype(np.float32) * 0.1
    mask = (rng.random(T) < 0.9).astype(np.uint8)
    x = _logits(rng, T, E, torch.float32)
    _check(gpu_lib, x, min(k, keep * (E // G)), score, bias=bias, num_groups=G, topk_groups=keep, group_top=2 if G > 1 else 1,
           mask=mask, renormalize=False)
    # the same rows in a small batch: the same choice
    ids, _ = gpu_lib.mx_moe_route(x.cuda(), k, score=score)
    few, _ = gpu_lib.mx_moe_route(x[-99:].cuda(), k, score=score)
    assert torch.equal(ids[-99:], few)


def _sizes(x, ids, g, softmax, renorm):
    """Bound of the terms of each logit's gradient."""
    out = np.zeros(x.shape)
    for t in range(x.shape[0]):
        r = x[t].astype(np.float64)
        s = np.exp(r - r.max()) / np.exp(r - r.max()).sum() if softmax else 1 / (1 + np.exp(-r))
        sel = ids[t]
        top = np.abs(g[t]).max() * 2
        if renorm:
            out[t, sel] = top * s[sel] / s[sel].sum()
        elif softmax:
            out[t] = top * s
        else:
            out[t, sel] = top * s[sel]
    return out


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,keep,gt", [(37, 64, 6, 8, 3, 1), (21, 256, 8, 8, 4, 2), (10, 60, 4, 20, 2, 2),
                                             (5, 1024, 8, 64, 5, 2), (9, 12, 4, 3, 2, 1), (4, 63, 3, 63, 3, 1)])
def test_groups_and_bias(gpu_lib, T, E, k, G, keep, gt, score):
    rng = np.random.default_rng(E + k)
    for bias in (None, rng.standard_normal(E).astype(np.float32) * 0.1):
        _check(gpu_lib, _logits(rng, T, E, torch.float32), k, score, bias=bias, num_groups=G, topk_groups=keep,
               group_top=gt, scale=2.5)


def test_ties_go_to_the_lowest_expert(gpu_lib):
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.integers(-2, 3, (200, 96)).astype(np.float32))
    x[0] = 0.0
    x[1] = -0.0
    x[2, ::2] = -0.0
    for score in ("softmax", "sigmoid"):
        _check(gpu_lib, x, 8, score)
        _check(gpu_lib, x.bfloat16(), 8, score, bias=np.zeros(96, np.float32))
        _check(gpu_lib, x, 8, score, num_groups=8, topk_groups=3, group_top=2)
        # far out both scores saturate; the logits still order the experts
        _check(gpu_lib, x * 30, 8, score)


def test_rows_with_nothing_left(gpu_lib):
    """-inf experts, whole rows of them, masked tokens: ids -1, weights and gradients 0."""
    mx = gpu_lib
    rng = np.random.default_rng(6)
    T, E, k = 40, 64, 6
    x = _logits(rng, T, E, torch.float32)
    x[0] = -np.inf
    x[1, 3:] = -np.inf           # three left
    x[2] = torch.finfo(torch.float32).min
    x[3, 10] = torch.finfo(torch.float32).max / 4
    x[4] = -95.0                 # every sigmoid underflows in FP32
    x[4, 7] = -94.0
    mask = (rng.random(T) < 0.7).astype(np.uint8)
    mask[:5] = 1
    xm = x.clone()
    xm[torch.from_numpy(mask == 0)] = float("nan")   # a masked token's logits are not read
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            T_ = slice(0, T)
            ids, w = mx.mx_moe_route(xm.cuda(), k, score=score, renormalize=renorm, mask=torch.from_numpy(mask).cuda())
            rid, rw = ref.route(x.numpy(), k, score == "softmax", renorm=renorm, mask=mask)
            assert np.array_equal(ids.cpu().numpy()[T_], rid)
            fine = np.ones(T, bool)
            fine[[2, 3, 4]] = False      # their values are checked below
            e = np.abs(w.cpu().numpy() - rw)[fine]
            assert (e <= 128 * U * rw[fine] + 1e-44).all()
            assert (w[0] == 0).all() and (ids[0] == -1).all() and (ids[1, 3:] == -1).all() and (w[1, 3:] == 0).all()
            assert torch.isfinite(w).all()
            if renorm:
                assert torch.allclose(w[[2, 4]].sum(1).cpu(), torch.ones(2), atol=1e-6)
            g = torch.randn(T, k, device="cuda")
            dx = mx.mx_moe_route_bwd(g, x.cuda(), ids, score=score, renormalize=renorm)
            assert (dx[0] == 0).all() and torch.isfinite(dx).all()
            assert (dx[1, 3:] == 0).all()
            assert (dx[torch.from_numpy(mask == 0).cuda()] == 0).all()
    # all groups but one masked out
    y = x.clone()
    y[:, 8:] = -np.inf
    ids, w = mx.mx_moe_route(y.cuda(), 12, num_groups=8, topk_groups=2, group_top=1)
    assert (ids[5:, 8:] == -1).all() and (ids[5:, :8].sort(1).values == torch.arange(8, device="cuda")).all()


def test_nan_and_inf_stay_in_range(gpu_lib):
    mx = gpu_lib
    rng = np.random.default_rng(8)
    x = _logits(rng, 12, 40, torch.float32)
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    x[3] = float("nan")
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(40, device="cuda")):
            ids, w = mx.mx_moe_route(x.cuda(), 4, score=score, bias=bias)
            assert ((ids >= 0) & (ids < 40)).all()
            assert torch.isnan(w[1]).any() and torch.isnan(w[3]).all()
            if bias is None:
                assert ids[1, 0] == 7 and ids[2, 0] == 9
            keep = [0, 4, 5, 6, 7, 8, 9, 10, 11]
            assert torch.isfinite(w[keep]).all()
            dx = mx.mx_moe_route_bwd(torch.ones(12, 4, device="cuda"), x.cuda(), ids, score=score)
            assert torch.isfinite(dx[keep]).all()


def test_gradient_against_differences(gpu_lib):
    """Central differences of the kernel's own weights.  Logits are distinct
    multiples of 1/4, so a step of 2^-6 does not change the choice; the
    truncation error is below h^2 (2^-12) of third derivatives of size one
    and the rounding below 2^-22 / h."""
    mx = gpu_lib
    rng = np.random.default_rng(9)
    T, E, k, h = 6, 24, 4, 2.0 ** -6
    x = torch.from_numpy(np.stack([rng.permutation(E) for _ in range(T)]).astype(np.float32) / 4 - 3).cuda()
    g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            how = dict(score=score, renormalize=renorm, scale=1.0)
            ids, _ = mx.mx_moe_route(x, k, **how)
            dx = mx.mx_moe_route_bwd(g, x, ids, **how)
            num = torch.zeros_like(x)
            for e in range(E):
                d = torch.zeros_like(x)
                d[:, e] = h
                lp = (mx.mx_moe_route(x + d, k, **how)[1] * g).sum(1)
                lm = (mx.mx_moe_route(x - d, k, **how)[1] * g).sum(1)
                num[:, e] = (lp - lm) / (2 * h)
            assert (num - dx).abs().max() <= 2.0 ** -12 * 8 * g.abs().max() + 2.0 ** -22 / h * 8


def test_route_strides_outputs_and_repeated_ids(gpu_lib):
    mx = gpu_lib
    rng = np.random.default_rng(10)
    T, E, k = 50, 70, 5
    wide = torch.full((T, 101), float("nan"))
    x = _logits(rng, T, E, torch.float32)
    wide[:, 3:3 + E] = x
    view = wide.cuda()[:, 3:3 + E]
    ids, w = mx.mx_moe_route(view, k)
    ids2, w2 = mx.mx_moe_route(x.cuda(), k)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    out = torch.full((T, 90), 7.0, device="cuda")
    dx = mx.mx_moe_route_bwd(g, view, ids, d_logits=out[:, 1:1 + E])
    assert dx.data_ptr() == out[:, 1:].data_ptr()
    assert (out[:, 0] == 7).all() and (out[:, 1 + E:] == 7).all()
    assert torch.equal(out[:, 1:1 + E], mx.mx_moe_route_bwd(g, x.cuda(), ids))
    # ids that stand twice count twice, ids out of range not at all
    twice = ids.clone()
    twice[:, 1] = twice[:, 0]
    twice[:, 2] = E
    twice[:, 3] = -5
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            d = mx.mx_moe_route_bwd(g, x.cuda(), twice, score=score, renormalize=renorm)
            want = ref.route_bwd(x.numpy(), twice.cpu().numpy(), g.cpu().numpy(), score == "softmax", renorm)
            assert np.abs(d.cpu().numpy() - want).max() <= 256 * U * np.abs(g.cpu().numpy()).max() * 4


def test_route_empty_and_deterministic(gpu_lib):
    mx = gpu_lib
    ids, w = mx.mx_moe_route(torch.empty((0, 16), device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    d = mx.mx_moe_route_bwd(w, torch.empty((0, 16), device="cuda"), ids)
    assert d.shape == (0, 16)
    x = torch.randn(3000, 128, device="cuda")
    a = mx.mx_moe_route(x, 8, score="sigmoid", bias=torch.randn(128, device="cuda"))
    b = mx.mx_moe_route(x, 8, score="sigmoid", bias=torch.randn(128, device="cuda") * 0)
    assert not torch.equal(a[0], b[0])
    for _ in range(3):
        c = mx.mx_moe_route(x, 8)
        e = mx.mx_moe_route(x, 8)
        assert torch.equal(c[0], e[0]) and torch.equal(c[1], e[1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(37, 40, 3), (50, 128, 8), (41, 256, 17), (19, 1000, 8), (4301, 128, 8), (2303, 512, 4)])
def test_gradient_of_masked_rows(gpu_lib, T, E, k, score):
    """A masked token's logits may hold anything: its gradient is zero, that of
    the other rows the one they have alone.  So for rows of -inf alone."""
    mx = gpu_lib
    rng = np.random.default_rng(T + E)
    mask = torch.from_numpy((rng.random(T) < 0.6).astype(np.uint8)).cuda()
    mask[:6] = 0
    mask[6] = 1
    for dtype in (torch.float32, torch.bfloat16):
        clean = _logits(rng, T, E, dtype).cuda()
        clean[6] = -float("inf")
        x = clean.clone()
        x[mask == 0] = float("nan")
        x[1], x[2], x[3, 5], x[4] = float("inf"), -float("inf"), float("inf"), 0.0
        g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
        live = mask == 1
        for renorm in (True, False):
            how = dict(score=score, renormalize=renorm, scale=1.5)
            ids, w = mx.mx_moe_route(x, k, mask=mask, **how)
            assert (ids[~live] == -1).all() and (w[~live] == 0).all() and (ids[6] == -1).all()
            dx = mx.mx_moe_route_bwd(g, x, ids, **how)
            assert (dx[~live] == 0).all() and (dx[6] == 0).all() and torch.isfinite(dx).all()
            assert torch.equal(dx[live], mx.mx_moe_route_bwd(g, clean, ids, **how)[live])


@pytest.mark.parametrize("T,E,G,bias", [(9, 32, 4, False), (9, 256, 8, True), (5, 60, 20, True), (3, 1024, 64, False),
                                        (4301, 128, 8, True)])
def test_groups_of_two_with_experts_missing(gpu_lib, T, E, G, bias):
    """group_top 2 where -inf leaves a group one expert or none: groups of two
    and more first, then those of one by its score, empty ones last, so that a
    token keeps an expert as long as one can be chosen."""
    mx = gpu_lib
    size = E // G
    b = torch.linspace(-0.4, 0.4, E).cuda() if bias else None
    x = torch.full((T, E), -float("inf"))
    x[:, E - 1] = -3.0                                  # the last group alone has an expert
    for score in ("softmax", "sigmoid"):
        how = dict(score=score, bias=b, num_groups=G, group_top=2)
        ids, w = mx.mx_moe_route(x.cuda(), 2, topk_groups=1, **how)
        assert (ids[:, 0] == E - 1).all() and (ids[:, 1] == -1).all()
        assert (w[:, 0] == 1).all() and (w[:, 1] == 0).all()
        y = x.clone()
        y[:, size] = 4.0                                # group 1: one expert of a larger score
        ids, _ = mx.mx_moe_route(y.cuda(), 2, topk_groups=1, **how)
        assert (ids[:, 0] == size).all() and (ids[:, 1] == -1).all()
        ids, _ = mx.mx_moe_route(y.cuda(), 2, topk_groups=2, **how)
        assert (ids[:, 0] == size).all() and (ids[:, 1] == E - 1).all()
        y[:, 2 * size:2 * size + 2] = -3.0              # group 2: two of smaller ones
        ids, _ = mx.mx_moe_route(y.cuda(), 2, topk_groups=1, **how)
        assert (ids.sort(1).values == torch.tensor([2 * size, 2 * size + 1]).cuda()).all()
        ids, _ = mx.mx_moe_route(y.cuda(), 4, topk_groups=3, **how)
        assert (ids[:, 0] == size).all()
        assert (ids.sort(1).values == torch.tensor([size, 2 * size, 2 * size + 1, E - 1]).cuda()).all()
        ids, w = mx.mx_moe_route(torch.full_like(x, -float("inf")).cuda(), 2, topk_groups=1, **how)
        assert (ids == -1).all() and (w == 0).all()


@pytest.mark.parametrize("E", [32, 128, 256, 1024])
def test_order_of_nan_and_inf(gpu_lib, E):
    """Logits compared: NaN, then +inf, then numbers.  Scores compared: a softmax
    row with either ranks by its logits in that order, the bias left out; with
    sigmoid NaN is first and +inf has the score 1."""
    mx = gpu_lib
    nan, inf = float("nan"), float("inf")
    x = torch.linspace(-2, 2, E).repeat(3, 1)
    x[0, 9], x[0, 3] = nan, inf
    x[1, 3] = inf
    x[2, 9] = nan
    bias = torch.zeros(E)
    bias[20], bias[9] = 5.0, -5.0
    top = E - 1
    for score in ("softmax", "sigmoid"):
        ids = mx.mx_moe_route(x.cuda(), 3, score=score)[0].cpu()
        assert ids.tolist() == [[9, 3, top], [3, top, top - 1], [9, top, top - 1]]
    ids = mx.mx_moe_route(x.cuda(), 3, bias=bias.cuda())[0].cpu()
    assert ids.tolist() == [[9, 3, top], [3, top, top - 1], [9, top, top - 1]]
    ids = mx.mx_moe_route(x.cuda(), 3, score="sigmoid", bias=bias.cuda())[0].cpu()
    assert ids.tolist() == [[9, 20, 3], [20, 3, top], [9, 20, top]]
    # groups of the same: one that holds a NaN ranks above one of two +inf
    y = torch.linspace(-2, 2, E).repeat(2, 1)
    y[0, :2], y[0, E // 4] = inf, nan
    y[1, :2], y[1, E // 4 + 1] = inf, 1.0
    ids = mx.mx_moe_route(y.cuda(), 1, num_groups=4, topk_groups=1, group_top=2)[0].cpu()
    assert ids.tolist() == [[E // 4], [0]]


# ---------------------------------------------------------------------------
# the combine's gradient


@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (1, 2048, 8), (5, 64, 3), (33, 520, 8), (17, 1024, 9), (40, 2048, 8),
                                   (11, 4104, 20), (300, 256, 2), (3, 7168, 8), (514, 2056, 3)])
def test_combine_bwd(gpu_lib, T, H, k):
    mx = gpu_lib
    rng = np.random.default_rng(T + H + k)
    n = T * k
    slot = rng.permutation(n).astype(np.int32)
    slot[rng.random(n) < 0.1] = -1
    if n > 4:
        slot[2] = n + 3       # not a row: skipped
    w = rng.standard_normal((T, k)).astype(np.float32)
    y = mxsynth.normal_bf16((n, H), 1.0, seed=1)
    d = mxsynth.normal_bf16((T, H), 1e-2, seed=2)
    for row in range(n):      # rows of y that no slot names are never read into a result
        if row not in slot:
            y[row] = float("nan")
    ld = H + 24
    dyb = torch.full((n, ld), 3.0, dtype=torch.bfloat16, device="cuda")
    dy, dw = mx.mx_moe_combine_bwd(d.cuda(), y.cuda(), torch.from_numpy(slot).cuda(), torch.from_numpy(w).cuda(),
                                   dy=dyb[:, :H])
    torch.cuda.synchronize()
    want = torch.full((n, H), 3.0, dtype=torch.bfloat16)
    ok = (slot >= 0) & (slot < n)
    prod = (torch.from_numpy(w)[:, :, None] * d.float()[:, None]).bfloat16().view(n, H)
    want[torch.from_numpy(slot[ok].astype(np.int64))] = prod[torch.from_numpy(ok)]
    assert torch.equal(dy.cpu().view(torch.int16), want.view(torch.int16))     # one rounding each: exact
    assert (dyb[:, H:] == 3.0).all()
    dn, yn = d.double().numpy(), y.double().numpy()
    got = dw.cpu().numpy().reshape(-1)
    for a in range(n):
        if not ok[a]:
            assert got[a] == 0
            continue
        p = dn[a // k] * yn[slot[a]]
        # any order of H fused additions
        assert abs(got[a] - p.sum()) <= H * U * np.abs(p).sum() + 1e-38
    only, none = mx.mx_moe_combine_bwd(d.cuda(), None, torch.from_numpy(slot).cuda(), torch.from_numpy(w).cuda(),
                                       want_d_weights=False)
    assert none is None
    keep = torch.from_numpy(slot[ok].astype(np.int64))
    assert torch.equal(only.cpu()[keep], want[keep])
    none, dw2 = mx.mx_moe_combine_bwd(d.cuda(), y.cuda(), torch.from_numpy(slot).cuda(), torch.from_numpy(w).cuda(),
                                      want_dy=False)
    assert none is None and torch.equal(dw, dw2)


def test_combine_bwd_empty(gpu_lib):
    mx = gpu_lib
    bf = dict(dtype=torch.bfloat16, device="cuda")
    dy, dw = mx.mx_moe_combine_bwd(torch.empty((0, 64), **bf), torch.empty((0, 64), **bf),
                                   torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty((0, 4), device="cuda"))
    assert dy.shape == (0, 64) and dw.shape == (0, 4)
    # no columns: the dot products are zero
    dw = mx.mx_moe_combine_bwd(torch.empty((3, 0), **bf), torch.empty((6, 0), **bf),
                               torch.arange(6, dtype=torch.int32, device="cuda"), torch.ones((3, 2), device="cuda"))[1]
    assert (dw == 0).all()
