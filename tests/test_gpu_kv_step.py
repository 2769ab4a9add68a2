"""A sampler's attention step as it is used: queries rotated, keys and values appended, attention, token by
token against the 64-bit loops; the same step captured once and replayed as the sequences grow; on several
streams at once; and beside the rest of a layer (qkv projection by mx_gemm_fp4)."""
import numpy as np
import pytest
import torch

import kv_ref as ref
from kv_util import BF, Batch, bf16, check_attention

pytestmark = pytest.mark.gpu

HQ, HK, D = 8, 2, 64


def _freqs(mx, dev="cuda"):
    return mx.mx_rope_frequencies(D, 1e6, "yarn", 4.0, 4096, device=dev)


class Step:
    """One step's buffers; run() makes its calls."""

    def __init__(self, mx, B, qkv, dev="cuda", max_new=0):
        self.mx, self.qkv, self.max_new = mx, qkv, max_new
        self.freqs, self.amp = _freqs(mx, dev)
        self.kv, self.scale, self.table, self.lens, self.starts = (t.to(dev) for t in B.args)
        rows = qkv.shape[0]
        self.pos = torch.zeros(rows, dtype=torch.int32, device=dev)
        self.q = torch.empty(rows, HQ, D, dtype=BF, device=dev)
        self.out = torch.zeros(rows, HQ, D, dtype=BF, device=dev)
        self.lse = torch.zeros(rows, HQ, device=dev)
        need = mx.mx_kv_attention_workspace_bytes(rows, len(B.new), HQ, HK, D, max_new)
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)

    def run(self, stream=None):
        mx, kw = self.mx, dict(amplitude=self.amp, stream=stream)
        qkv = self.qkv
        cache = (self.kv, self.scale, self.table, self.lens)
        mx.mx_rope(qkv[:, :HQ], self.pos, self.freqs, y=self.q, **kw)
        mx.mx_kv_append(qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:], *cache, self.starts, freqs=self.freqs, **kw)
        mx.mx_kv_attention(self.q, *cache, self.starts, max_new=self.max_new, out=self.out, lse=self.lse, workspace=self.ws,
                           stream=stream)


def _check(mx, S, B, pos):
    """S.out against the loops, B.ref advanced by the step's rows."""
    x = S.qkv.double().cpu().numpy()
    f = S.freqs.cpu().numpy()
    n = int(B.starts[-1])
    q = ref.rope(x[:n, :HQ], pos[:n], f, amplitude=S.amp)
    got_q = S.q.double().cpu().numpy()[:n]
    # rounded to BF16 once, FP32 before: half a step and 5 roundings of the pair's magnitude
    pair = np.abs(x[:n, :HQ])
    pair = np.concatenate([pair[..., :D // 2] + pair[..., D // 2:]] * 2, -1) * S.amp
    assert (np.abs(got_q - q) <= 2.0 ** -8 * np.abs(q) + 6 * 2.0 ** -24 * pair).all()
    B.ref.append(x[:n, HQ:HQ + HK], x[:n, HQ + HK:], B.starts, B.lens, f, amplitude=S.amp)
    assert np.array_equal(S.kv.cpu().numpy(), B.ref.kv) and np.array_equal(S.scale.cpu().numpy(), B.ref.scale)
    check_attention(S.out[:n], S.lse[:n], B.ref.attention(got_q, B.starts, B.lens, D ** -0.5), D, int(max(B.lens.max(), 1)))


def _pos(B):
    return np.concatenate([np.arange(l - n, l) for n, l in zip(B.new, B.lens)] + [[0] * (B.rows - int(B.starts[-1]))]).astype(np.int32)


def test_prompt_then_tokens(gpu_lib):
    """A ragged prompt, then five tokens a sequence."""
    mx = gpu_lib
    B = Batch(50, [35, 1, 90], [0, 0, 0], HK, D, 16, spare=12, filled=False)
    free = [p for p in range(B.kv.shape[1]) if p not in B.table]
    B.table[:, -1] = free[:3]
    S = Step(mx, B, bf16(B.rng, B.rows, HQ + 2 * HK, D).cuda())
    S.pos.copy_(torch.from_numpy(_pos(B)))
    S.run()
    torch.cuda.synchronize()
    _check(mx, S, B, _pos(B))
    B.new, B.starts, B.rows = [1, 1, 1], np.arange(4, dtype=np.int64), 3
    # the table has to reach the new positions
    for b in range(3):
        used = -(-int(B.lens[b]) // 16)
        if used < B.table.shape[1] and B.table[b, used] < 0:
            B.table[b, used] = free[3 + b]
    B.ref.table = B.table
    kv, scale = S.kv, S.scale
    for step in range(5):
        B.lens += 1
        T = Step(mx, B, bf16(B.rng, 3, HQ + 2 * HK, D).cuda(), max_new=1)
        T.kv, T.scale = kv, scale
        T.pos.copy_(torch.from_numpy(_pos(B)))
        T.run()
        torch.cuda.synchronize()
        _check(mx, T, B, _pos(B))


@pytest.mark.parametrize("max_new,room", [(1, 0), (0, 0), (1, 1500), (0, 1500)])
def test_a_captured_step_follows_growing_sequences(gpu_lib, max_new, room):
    """Captured once; every replay finds longer sequences, other rows, some without a new one (a padded batch)."""
    mx = gpu_lib
    B = Batch(51 + max_new, [1] * 6, [0, 14, 15, 40, 130, 3], HK, D, 16, spare=8, filled=True, room=room)
    B.table[:, 9] = [p for p in range(B.kv.shape[1]) if p not in B.table][:6]
    B.ref.table = B.table
    S = Step(mx, B, bf16(B.rng, 8, HQ + 2 * HK, D).cuda(), max_new=max_new)
    B.rows = 8
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    lens0 = B.lens.copy()
    S.lens.zero_()  # (nothing is stored while it is captured)
    S.starts.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        S.run()
    B.lens = lens0
    for step in range(5):
        B.new = [1] * 6 if step % 2 == 0 else [1, 0, 1, 1, 0, 1]
        if step:
            B.lens = B.lens + np.array(B.new, np.int32)
        B.starts = np.concatenate([[0], np.cumsum(B.new)]).astype(np.int64)
        S.starts.copy_(torch.from_numpy(B.starts))
        S.lens.copy_(torch.from_numpy(B.lens))
        S.table.copy_(torch.from_numpy(B.table))
        S.pos.copy_(torch.from_numpy(_pos(B)))
        S.qkv.copy_(bf16(B.rng, 8, HQ + 2 * HK, D))
        S.out.fill_(5.0)
        S.ws.random_(0, 256)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _check(mx, S, B, _pos(B))
        assert (S.out[int(B.starts[-1]):] == 5.0).all()
        torch.ones(1000, device="cuda").sum().item()  # the program's own work between replays


def test_two_graphs_and_eager_work_share_nothing_but_what_they_are_given(gpu_lib):
    """Two captured steps on their own caches and workspaces, replayed at the same time."""
    mx = gpu_lib
    steps, want, graphs, streams = [], [], [], []
    for i in range(2):
        B = Batch(60 + i, [1, 40, 3], [300, 0, 61], HK, D, 32, spare=4, room=1500)
        S = Step(mx, B, bf16(B.rng, B.rows, HQ + 2 * HK, D).cuda())
        S.pos.copy_(torch.from_numpy(_pos(B)))
        S.run()
        S.run()  # (the codes of a block's older rows have settled)
        torch.cuda.synchronize()
        want.append((S.out.clone(), S.lse.clone(), S.kv.clone(), S.scale.clone()))
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            S.run()
        steps.append(S)
        graphs.append(g)
        streams.append(s)
    for rep in range(3):
        for S in steps:
            S.out.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for S, w in zip(steps, want):
            assert torch.equal(S.out, w[0]) and torch.equal(S.lse, w[1]) and torch.equal(S.kv, w[2]) and torch.equal(S.scale, w[3])


def test_streams(gpu_lib):
    """Steps on two streams at once, one given by stream=, equal the same steps one after the other."""
    mx = gpu_lib
    B = [Batch(70 + i, [1, 1, 70], [200, 5, 33], HK, D, 64, room=1500) for i in range(2)]
    qkv = [bf16(b.rng, b.rows, HQ + 2 * HK, D).cuda() for b in B]
    S = [Step(mx, b, x) for b, x in zip(B, qkv)]
    for s, b in zip(S, B):
        s.pos.copy_(torch.from_numpy(_pos(b)))
        s.run()
        s.run()
    torch.cuda.synchronize()
    want = [(s.out.clone(), s.kv.clone()) for s in S]
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        for s in S:
            s.out.zero_()
        torch.cuda.synchronize()
        S[0].run(stream=st[0])
        S[1].run(stream=st[1].cuda_stream)
        torch.cuda.synchronize()
        for s, w in zip(S, want):
            assert torch.equal(s.out, w[0]) and torch.equal(s.kv, w[1])
    # outputs and workspaces that the call makes belong to its stream
    out = mx.mx_kv_attention(S[0].q, S[0].kv, S[0].scale, S[0].table, S[0].lens, S[0].starts, stream=st[1])
    st[1].synchronize()
    assert torch.equal(out, want[0][0])


def test_after_a_projection(gpu_lib):
    """The step on what the library's MXFP4 projection gives, straight from its output."""
    mx = gpu_lib
    H, rows = 256, 5
    B = Batch(80, [1] * rows, [20, 0, 15, 100, 31], HK, D, 32)
    x, w = bf16(B.rng, rows, H).cuda(), bf16(B.rng, (HQ + 2 * HK) * D, H, std=0.1).cuda()
    qkv = mx.mx_gemm_fp4(*mx.mx_quantize_rowwise_fp4(x), *mx.mx_quantize_rowwise_fp4(w)).view(rows, HQ + 2 * HK, D)
    S = Step(mx, B, qkv, max_new=1)
    S.pos.copy_(torch.from_numpy(_pos(B)))
    S.run()
    torch.cuda.synchronize()
    _check(mx, S, B, _pos(B))


def _fresh(S, before, qkv):
    """The step's buffers as before its append, with other rows; whatever a step leaves is garbage."""
    S.kv.copy_(before[0])
    S.scale.copy_(before[1])
    S.qkv.copy_(qkv)
    S.q.fill_(9.0)
    S.out.fill_(5.0)
    S.lse.fill_(float("nan"))
    S.ws.fill_(255)


def _left(S):
    return [t.clone() for t in (S.q, S.kv, S.scale, S.out, S.lse)]


@pytest.mark.parametrize("captured", [False, True])
def test_two_steps_at_once_from_fresh_buffers(gpu_lib, captured):
    """Two steps on two streams, eager or replayed, on other rows every time and from the cache as it was: each of their
    three calls has to run, in its order, for the bytes of the same steps one after the other."""
    mx = gpu_lib
    B = [Batch(90 + i, [1, 1, 70], [200, 5, 33], HK, D, 64, room=1500) for i in range(2)]
    S = [Step(mx, b, bf16(b.rng, b.rows, HQ + 2 * HK, D).cuda()) for b in B]
    before = [(s.kv.clone(), s.scale.clone()) for s in S]
    for s, b in zip(S, B):
        s.pos.copy_(torch.from_numpy(_pos(b)))
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = []
    if captured:
        for s, stream in zip(S, st):
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=stream):
                s.run()
            graphs.append(g)
    last = None
    for rep in range(3):
        rows = [bf16(b.rng, b.rows, HQ + 2 * HK, D).cuda() for b in B]
        want = []
        for s, w, x in zip(S, before, rows):
            _fresh(s, w, x)
            s.run()
            torch.cuda.synchronize()
            want.append(_left(s))
        assert last is None or not torch.equal(want[0][3], last)
        last = want[0][3]
        for s, w, x in zip(S, before, rows):
            _fresh(s, w, x)
        torch.cuda.synchronize()
        for i in range(2):
            if captured:
                with torch.cuda.stream(st[i]):
                    graphs[i].replay()
            else:
                S[i].run(stream=st[i])
        torch.cuda.synchronize()
        for s, w in zip(S, want):
            for a, b in zip(_left(s), w):
                assert torch.equal(a, b)
        assert all(torch.isfinite(w[3].float()).all() and torch.isfinite(w[4]).all() for w in want)
