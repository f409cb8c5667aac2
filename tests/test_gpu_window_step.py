"""A sliding-window model's serving steps through the public calls, as an engine makes them: tables built on the GPU,
query and key rows normalised and rotated on the way into the cache, windowed attention of chunks and of single tokens,
blocks given back; against 64-bit sums over the whole history, kept outside the cache."""
import numpy as np
import pytest
import torch

import paged_kv_cache_slots_gb300 as pkv

pytestmark = pytest.mark.gpu
H, KV, D, BS = 8, 2, 128, 16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    torch.cuda.empty_cache()


class Engine:
    def __init__(self, B, NB, dtype=torch.bfloat16, window=50, sinks=4, cache=None, max_blocks=64, seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.window, self.sinks, self.dtype = B, window, sinks, dtype
        self.pool = pkv.KVPool(1, NB, BS, KV, D, cache or dtype)
        self.pool.buffer.fill_(0xFF)  # NaN in every type
        self.scales = dict(k_scale=1 / 64, v_scale=1 / 44) if cache else {}
        self.freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        self.rope = pkv.Rope(self.freq)
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=self.g, device="cuda")).to(dtype) for _ in range(2))
        self.tables = torch.full((B, max_blocks), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.queue, self.state = pkv.make_free_queue(NB, device="cuda")
        self.history = [[] for _ in range(B)]  # of each sequence: rows (k after norm and rotation, v) in float64

    def rows(self, T):
        return torch.randn((T, H + 2 * KV, D), generator=self.g, device="cuda").to(self.dtype)

    def launch(self, qkv, new, o, q_out, out, ws, decode):
        """The step's calls, nothing else (what a graph captures)."""
        T = qkv.shape[0]
        pkv.extend_tables(self.tables, self.lens, new, self.queue, self.state, BS, T, out=o)
        self.pool.append_norm_rope(0, qkv[:, H:H + KV], qkv[:, H + KV:], o.slot_mapping, o.positions, self.rope, self.kw, q=qkv[:, :H],
                                   q_weight=self.qw, eps=EPS, q_out=q_out, seq_ids=o.seq_ids, **self.scales)
        kc, vc = self.pool.layer(0)
        if decode:
            pkv.paged_window_decode_attention(q_out, kc, vc, self.tables, o.context_lens, D ** -0.5, self.window, self.sinks, out=out,
                                              workspace=ws, **self.scales)
        else:
            pkv.paged_window_prefill_attention(q_out, kc, vc, self.tables, o.query_start, o.context_lens, D ** -0.5, self.window,
                                               self.sinks, out=out, workspace=ws, **self.scales)

    def buffers(self, T, decode):
        o = pkv.make_step_tables(self.B, T)._replace(context_lens=self.lens, queue_state=self.state)
        q_out = torch.zeros((T, H, D), dtype=self.dtype, device="cuda")
        ws = (pkv.make_workspace(self.B, H, KV, D) if decode else pkv.make_window_prefill_workspace(self.B, T, H, KV, D))
        return o, q_out, torch.zeros_like(q_out), ws

    def turned(self, x, w, pos):
        x = x.double()
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
        t = pos.double()[:, None, None] * self.freq.cuda()
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat((a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()), -1)

    def check(self, qkv, o, out):
        """The step's rows of out against the history; the new rows join it."""
        assert pkv.device_status() == (0, 0)
        pos, ids = o.positions, o.seq_ids.tolist()
        q = self.turned(qkv[:, :H], self.qw, pos)
        k, v = self.turned(qkv[:, H:H + KV], self.kw, pos), qkv[:, H + KV:].double()
        for t, s in enumerate(ids):
            if s < 0:
                continue
            assert pos[t].item() == len(self.history[s])
            self.history[s].append((k[t], v[t]))
            n = len(self.history[s])
            seen = [j for j in range(n) if j > n - 1 - self.window or j < self.sinks]
            kk, vv = (torch.stack([self.history[s][j][i] for j in seen], 1) for i in (0, 1))  # [KV, n, D]
            p = torch.softmax(q[t].view(KV, H // KV, D) @ kk.mT * D ** -0.5, -1)
            ref = (p @ vv).view(H, D)
            # Rounding of q and k (half a step each) moves a score by eps |q| |k| scale at most, so a weight by twice that
            # relatively; a cached V is off by half a step of its type, the output and the weights by half a step of theirs.
            half = 2.0 ** -4 if self.scales else torch.finfo(self.dtype).eps / 2
            step = torch.finfo(self.dtype).eps / 2
            err = (step + half) * (q[t].view(KV, H // KV, D).abs() @ kk.abs().mT).amax(-1, keepdim=True) * D ** -0.5
            tol = (p @ vv.abs()) * (2 * err.expm1() + half + 2 * step + 2.0 ** -12)
            assert float(((out[t].double() - ref).abs() - tol.view(H, D)).max()) <= 0, (t, s, n)


@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, None), (torch.float16, None), (torch.float16, torch.float8_e4m3fn)])
def test_prompts_then_tokens(dtype, cache):
    e = Engine(4, 40, dtype, cache=cache)
    used = []
    for new in ([70, 1, 0, 33], [40, 90, 1, 1], [1, 1, 100, 1]):
        T = sum(new) + 5
        o, q_out, out, ws = e.buffers(T, False)
        qkv = e.rows(T)
        e.launch(qkv, torch.tensor(new, dtype=torch.int32, device="cuda"), o, q_out, out, ws, False)
        e.check(qkv, o, out)
        assert bool((out[sum(new):] == 0).all())
        pkv.release_tables(e.tables, e.lens, e.queue, e.state, BS, window=e.window, sinks=e.sinks)
    ones = torch.ones(4, dtype=torch.int32, device="cuda")
    o, q_out, out, ws = e.buffers(4, True)
    for step in range(60):
        qkv = e.rows(4)
        e.launch(qkv, ones, o, q_out, out, ws, True)
        if step % 7 == 0 or step > 55:
            e.check(qkv, o, out)
        else:
            k, v = e.turned(qkv[:, H:H + KV], e.kw, o.positions), qkv[:, H + KV:].double()
            for s in range(4):
                e.history[s].append((k[s], v[s]))
        pkv.release_tables(e.tables, e.lens, e.queue, e.state, BS, window=e.window, sinks=e.sinks)
        used.append(40 - e.state[1].item())
    # A window of 50 and 4 first tokens: one block of those and at most five of the window's a sequence, however long.
    assert max(used[4:]) <= 4 * 6
    assert pkv.device_status() == (0, 0)


def test_captured_decode_steps():
    """Tables, append, attention and release in one graph, replayed for many steps without the host."""
    e = Engine(3, 30, sinks=2, window=33)
    o, q_out, out, ws = e.buffers(140, False)
    qkv = e.rows(140)
    e.launch(qkv, torch.tensor([60, 50, 30], dtype=torch.int32, device="cuda"), o, q_out, out, ws, False)
    e.check(qkv, o, out)
    ones = torch.ones(3, dtype=torch.int32, device="cuda")
    o, q_out, out, ws = e.buffers(3, True)
    qkv = e.rows(3)
    pkv.release_tables(e.tables, e.lens, e.queue, e.state, BS, window=33, sinks=2)
    torch.cuda.synchronize()
    kept = [x.clone() for x in (e.tables, e.lens, e.queue, e.state, e.pool.buffer)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.launch(qkv, ones, o, q_out, out, ws, True)
        pkv.release_tables(e.tables, e.lens, e.queue, e.state, BS, window=33, sinks=2)
    for x, y in zip((e.tables, e.lens, e.queue, e.state, e.pool.buffer), kept):
        assert torch.equal(x, y)  # (capturing runs nothing)
    for _ in range(40):
        qkv.copy_(e.rows(3))
        g.replay()
        torch.cuda.synchronize()
        e.check(qkv, o, out)


def test_out_of_blocks_then_room_again():
    e = Engine(3, 6, max_blocks=8)
    qkv = e.rows(100)
    o, q_out, out, ws = e.buffers(100, False)
    e.launch(qkv, torch.tensor([40, 60, 10], dtype=torch.int32, device="cuda"), o, q_out, out, ws, False)  # 3, 4 and 1 blocks
    assert o.query_start.tolist() == [0, 40, 40, 40]
    e.check(qkv, o, out)
    assert bool((out[40:] == 0).all())
    pkv.release_tables(e.tables, e.lens, e.queue, e.state, BS, finished=torch.tensor([1, 0, 0], dtype=torch.int32, device="cuda"))
    e.history[0] = []
    e.launch(qkv, torch.tensor([0, 60, 10], dtype=torch.int32, device="cuda"), o, q_out, out, ws, False)
    assert o.query_start.tolist() == [0, 0, 60, 70]
    e.check(qkv, o, out)
    assert np.array_equal(e.state.cpu().numpy()[1:], [1])
