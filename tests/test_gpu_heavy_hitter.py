"""The calls as a program makes them: packed prompts are written and attended to,
their weights taken, the caches held to a budget, and decode steps run over what is
left, with an eviction every few steps.  Every step is checked against the
sequences' whole histories: what each slot holds is named by its position, and
the attention over those positions is recomputed in 64 bits."""
import numpy as np
import pytest
import torch

import evict_reference as ref
from paged_kv_cache_444_b200 import (EvictionState, PagedAttentionError, WeightsWorkspace,
                                     pa_check_error, pa_decode_weights, pa_evict_commit,
                                     pa_reshape_and_cache, prompt_step)
from weights_reference import HALF, attend, out_bound

pytestmark = pytest.mark.gpu
H, HK, D, G = 8, 2, 64, 4
LENS, BUDGET, SINK, RECENT = (70, 130, 33, 48), 48, 2, 10
STEPS, EVERY = 34, 8


class Run:
    def __init__(self, dev, dtype, graph):
        self.dev, self.dtype, self.graph = dev, dtype, graph
        self.g = torch.Generator(device=dev).manual_seed(11)
        self.S, self.scale = len(LENS), D ** -0.5
        need = [-(-(max(n, BUDGET) + EVERY) // 16) for n in LENS]
        self.tables = torch.full((self.S, max(need)), -1, dtype=torch.int32)
        perm = torch.randperm(sum(need), generator=torch.Generator().manual_seed(3)).to(torch.int32)
        at = 0
        for s, m in enumerate(need):
            self.tables[s, :m] = perm[at:at + m]
            at += m
        self.tables = self.tables.to(dev)
        self.kc = torch.full((sum(need), 16, HK, D), float("nan"), dtype=dtype, device=dev)
        self.vc = self.kc.clone()
        self.ctx = torch.tensor(LENS, dtype=torch.int32, device=dev)
        self.length = self.ctx.clone()
        self.state = EvictionState(self.S, HK, max(LENS) + EVERY, BUDGET, dev, SINK, RECENT)
        # histories: K and V of every position, and the weight each has received
        self.k = [None] * self.S
        self.v = [None] * self.S
        self.received = [None] * self.S

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device=self.dev).to(self.dtype)

    def slots(self, s, first, n):
        at = torch.arange(first, first + n, device=self.dev)
        return self.tables[s, at // 16].long() * 16 + at % 16

    def prompt(self):
        T = sum(LENS)
        q, k, v = self.normal(T, H, D), self.normal(T, HK, D), self.normal(T, HK, D)
        starts = torch.tensor(np.concatenate([[0], np.cumsum(LENS)]), dtype=torch.int32,
                              device=self.dev)
        slots = torch.cat([self.slots(s, 0, n) for s, n in enumerate(LENS)])
        out = prompt_step(q, k, v, self.kc, self.vc, slots, starts, self.scale,
                          weights=self.state.weights, window=max(LENS))
        torch.cuda.synchronize()
        for s, n in enumerate(LENS):
            b = int(starts[s])
            self.k[s], self.v[s] = k[b:b + n], v[b:b + n]
            self.received[s] = torch.zeros((HK, n), dtype=torch.float64, device=self.dev)
            for h in range(H):
                p, o, _, rel, pv = attend(q[b:b + n, h], k[b:b + n, h // G], v[b:b + n, h // G],
                                          self.scale, 0)
                lim = out_bound(o, pv, rel, n, 8.0, self.dtype, HALF[self.dtype])
                assert ((out[b:b + n, h].double() - o).abs() <= lim).all()
                self.received[s][h // G] += p.sum(0)

    def kept(self, s, kv):
        """Positions of the cached tokens, in slot order."""
        n = int(self.ctx[s])
        return ref.slot_positions(self.state.positions[s, kv].cpu().numpy(),
                                  int(self.state.recorded_lens[s]), int(self.length[s]), n)

    def check_cache(self):
        """Rows and weights of every slot are those of the position it names."""
        for s in range(self.S):
            n = int(self.ctx[s])
            at = torch.arange(n, device=self.dev)
            blk, row = self.tables[s, at // 16].long(), at % 16
            for kv in range(HK):
                pos = self.kept(s, kv)
                assert len(set(pos.tolist())) == n and pos.min() >= 0
                assert pos.max() < int(self.length[s])
                assert set(range(min(SINK, n))) <= set(pos.tolist())
                latest = range(max(0, int(self.length[s]) - RECENT), int(self.length[s]))
                assert set(latest) <= set(pos.tolist())
                idx = torch.as_tensor(pos, device=self.dev)
                assert torch.equal(self.kc[blk, row, kv], self.k[s][idx, kv])
                assert torch.equal(self.vc[blk, row, kv], self.v[s][idx, kv])
                want = self.received[s][kv][idx]
                got = self.state.weights[s, kv, :n].double()
                # each addition is off by the bound of weights_reference, below 2^-10 of
                # the term here, and by half a step of the sum
                assert ((got - want).abs() <= 2.0 ** -10 * want).all()

    def evict(self):
        w, p = self.state.weights.cpu().numpy(), self.state.positions.cpu().numpy()
        source, new = ref.select(w, p, self.state.recorded_lens.cpu().numpy(),
                                 self.length.cpu().numpy(), self.ctx.cpu().numpy(), BUDGET, SINK,
                                 RECENT)
        self.state.evict(self.kc, self.vc, self.tables, self.ctx, self.length)
        torch.cuda.synchronize()
        assert np.array_equal(self.state.source.cpu().numpy(), source)
        assert np.array_equal(self.ctx.cpu().numpy(), new)

    def decode(self):
        """Buffers of a decode step, captured once if `graph`."""
        self.q, self.nk, self.nv = (torch.empty((self.S, h, D), dtype=self.dtype, device=self.dev)
                                    for h in (H, HK, HK))
        self.out = torch.empty_like(self.q)
        self.slot = torch.empty(self.S, dtype=torch.int64, device=self.dev)
        # (kept: the captured graph writes to it at every replay)
        self.ws = WeightsWorkspace.for_call(self.q, self.kc, self.tables)

        def step():
            pa_reshape_and_cache(self.nk, self.nv, self.kc, self.vc, self.slot)
            pa_decode_weights(self.out, self.state.weights, self.ws, self.q, self.kc, self.vc,
                              self.tables, self.ctx, self.scale, 1)

        if not self.graph:
            return step
        captured = torch.cuda.CUDAGraph()
        self.slot.fill_(-1)
        with torch.cuda.graph(captured):
            step()
        return captured.replay


@pytest.mark.parametrize("dtype,graph", [(torch.bfloat16, False), (torch.float16, True)])
def test_prompt_evict_decode(dtype, graph, cuda_device):
    r = Run(cuda_device, dtype, graph)
    r.prompt()
    r.check_cache()
    r.evict()
    r.check_cache()
    step = r.decode()
    p_half = 2.0 ** -16 if dtype == torch.bfloat16 else 2.0 ** -11
    for i in range(STEPS):
        r.q.copy_(r.normal(r.S, H, D))
        r.nk.copy_(r.normal(r.S, HK, D))
        r.nv.copy_(r.normal(r.S, HK, D))
        r.slot.copy_(torch.cat([r.slots(s, int(r.ctx[s]), 1) for s in range(r.S)]))
        r.ctx += 1
        r.length += 1
        step()
        torch.cuda.synchronize()
        for s in range(r.S):
            r.k[s] = torch.cat([r.k[s], r.nk[s:s + 1]])
            r.v[s] = torch.cat([r.v[s], r.nv[s:s + 1]])
            r.received[s] = torch.nn.functional.pad(r.received[s], (0, 1))
            for kv in range(HK):
                idx = torch.as_tensor(r.kept(s, kv), device=r.dev)
                n = idx.numel()
                p, o, _, rel, pv = attend(r.q[s, kv * G:(kv + 1) * G], r.k[s][idx, kv],
                                          r.v[s][idx, kv], r.scale)
                lim = out_bound(o, pv, rel, n, 8.0, dtype, p_half)
                err = (r.out[s, kv * G:(kv + 1) * G].double() - o).abs()
                assert (err <= lim).all(), (i, s, kv, float((err / lim).max()))
                r.received[s][kv].index_add_(0, idx, p.sum(0))
        r.check_cache()
        if i % EVERY == EVERY - 1:
            r.evict()
            r.check_cache()
    pa_check_error()
    assert int(r.length[2]) - int(r.ctx[2]) > 0       # even the short prompt was evicted from


def test_state_is_graph_capturable(cuda_device):
    """select, compact and the two length copies as one captured graph, replayed
    on contents that differ each time."""
    S, W, B = 3, 60, 20
    state = EvictionState(S, 1, W, B, cuda_device, 1, 3)
    kc = torch.arange(S * 4 * 16, device=cuda_device).half().view(-1, 16, 1, 1).expand(
        -1, -1, 1, 64).contiguous()
    vc = kc.clone()
    tables = torch.arange(S * 4, dtype=torch.int32, device=cuda_device).view(S, 4)
    ctx = torch.tensor([60, 21, 20], dtype=torch.int32, device=cuda_device)
    length = ctx.clone()
    graph = torch.cuda.CUDAGraph()
    before = kc.clone()
    with torch.cuda.graph(graph):
        state.evict(kc, vc, tables, ctx, length)
    for seed in (1, 2):
        kc.copy_(before)
        vc.copy_(before)
        ctx.copy_(torch.tensor([60, 21, 20], dtype=torch.int32))
        state.recorded_lens.zero_()
        w = np.random.default_rng(seed).random((S, 1, W), dtype=np.float32)
        state.weights.copy_(torch.as_tensor(w))
        graph.replay()
        torch.cuda.synchronize()
        source, new = ref.select(w, np.zeros((S, 1, W), np.int32), [0] * S, [60, 21, 20],
                                 np.array([60, 21, 20]), B, 1, 3)
        assert np.array_equal(state.source.cpu().numpy(), source)
        assert ctx.tolist() == new.tolist() == state.recorded_lens.tolist()
        for s in range(S):
            n = int(new[s])
            rows = kc[tables[s].long(), :, 0, 0].flatten().float().cpu().numpy()[:n]
            assert np.array_equal(rows, s * 64 + source[s, 0, :n])
            assert np.array_equal(state.positions[s, 0, :n].cpu().numpy(), source[s, 0, :n])
    pa_check_error()


class Layer:
    """One layer's tensors of its own, from a seed: a step from packed prompts to a
    decode step over the evicted cache."""

    def __init__(self, dev, seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.lens = ((900, 33, 410), (1700,), (300,) * 7)[seed % 3]
        self.S, T, self.width = len(self.lens), sum(self.lens), max(self.lens)
        rand = lambda *s: torch.randn(s, generator=g, device=dev).bfloat16()
        self.q, self.k, self.v = rand(T, 16, 128), rand(T, 4, 128), rand(T, 4, 128)
        self.query = rand(self.S, 16, 128)
        starts = np.concatenate([[0], np.cumsum(self.lens)])
        blocks = -(-self.width // 16)
        self.tables = torch.arange(self.S * blocks, dtype=torch.int32, device=dev).view(self.S, -1)
        slots = np.concatenate([s * blocks * 16 + np.arange(n) for s, n in enumerate(self.lens)])
        self.slots = torch.as_tensor(slots, device=dev)
        self.starts = torch.tensor(starts, dtype=torch.int32, device=dev)
        self.length = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        self.kc = torch.zeros((self.S * blocks, 16, 4, 128), dtype=torch.bfloat16, device=dev)
        self.vc = torch.zeros_like(self.kc)
        self.ctx = self.length.clone()
        self.state = EvictionState(self.S, 4, self.width, 128, dev, 4, 20)
        self.ws = WeightsWorkspace.for_call(self.query, self.kc, self.tables)
        self.out, self.step = torch.zeros_like(self.q), torch.zeros_like(self.query)
        self.lse = torch.zeros((T, 16), device=dev)

    def run(self):
        self.ctx.copy_(self.length)
        self.state.recorded_lens.zero_()
        prompt_step(self.q, self.k, self.v, self.kc, self.vc, self.slots, self.starts, 0.09,
                    out=self.out, lse=self.lse, weights=self.state.weights, window=200)
        self.state.evict(self.kc, self.vc, self.tables, self.ctx, self.length)
        pa_decode_weights(self.step, self.state.weights, self.ws, self.query, self.kc, self.vc,
                          self.tables, self.ctx, 0.09, 0)

    def results(self):
        return [t.clone() for t in (self.out, self.lse, self.step, self.state.weights,
                                    self.state.positions, self.state.source, self.kc, self.ctx)]


def test_layers_at_once_on_streams_and_in_graphs(cuda_device):
    """Three layers one after another, then at the same time on a stream each, eager and as
    captured graphs: the same bits."""
    layers = [Layer(cuda_device, seed) for seed in range(3)]
    for layer in layers:
        layer.run()
    torch.cuda.synchronize()
    want = [layer.results() for layer in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    graphs = []
    for layer in layers:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            layer.run()
    for again in range(6):
        for layer, stream, graph in zip(layers, streams, graphs):
            with torch.cuda.stream(stream):
                if again % 2:
                    graph.replay()
                else:
                    layer.run()
        torch.cuda.synchronize()
        pa_check_error()
        for layer, bits in zip(layers, want):
            for got, ours in zip(layer.results(), bits):
                assert torch.equal(got, ours)


def test_evict_keeps_a_length_it_cannot_use(cuda_device):
    """A context past the state's columns, or below zero, is reported; its length and what is
    recorded of it stay, so that the sequence is evicted from once the length is right."""
    S, W, B = 4, 60, 20
    state = EvictionState(S, 2, W, B, cuda_device, 1, 3)
    g = torch.Generator(device=cuda_device).manual_seed(12)
    state.weights.copy_(torch.rand(state.weights.shape, generator=g, device=cuda_device))
    kc = torch.randn((S * 4, 16, 2, 64), generator=g, device=cuda_device).half()
    vc = kc * 2
    tables = torch.arange(S * 4, dtype=torch.int32, device=cuda_device).view(S, 4)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda_device)
    ctx, length = i32(60, 61, -2, 0), i32(60, 70, 30, 0)
    state.recorded_lens.copy_(i32(0, 7, 5, 7))
    state.positions[1:, :, :7] = 3 * torch.arange(7, dtype=torch.int32, device=cuda_device)
    kept = [t[1:3].clone() for t in (state.weights, state.positions)]
    rows = kc[4:12].clone()
    state.evict(kc, vc, tables, ctx, length)
    with pytest.raises(PagedAttentionError, match="context_len, index [12]"):
        pa_check_error()
    assert ctx.tolist() == [20, 61, -2, 0]
    assert state.recorded_lens.tolist() == [20, 7, 5, 0]
    for was, t in zip(kept, (state.weights, state.positions)):
        assert torch.equal(was, t[1:3])
    assert torch.equal(rows, kc[4:12])
    ctx.copy_(i32(20, 50, 20, 0))             # sequence 1: 10 of the tokens dropped by the user
    length.copy_(i32(60, 59, 30, 0))
    recorded = state.recorded_lens.cpu().numpy()
    source, new = ref.select(state.weights.cpu().numpy(), state.positions.cpu().numpy(), recorded,
                             length.cpu().numpy(), ctx.cpu().numpy(), B, 1, 3)
    state.evict(kc, vc, tables, ctx, length)
    torch.cuda.synchronize()
    pa_check_error()
    assert np.array_equal(state.source.cpu().numpy(), source)
    assert ctx.tolist() == new.tolist() == state.recorded_lens.tolist()


@pytest.mark.parametrize("S", [1, 127, 128, 129, 1000])
def test_commit_takes_the_new_lengths_that_there_are(S, cuda_device):
    rng = np.random.default_rng(S)
    ctx = rng.integers(-3, 50, S).astype(np.int32)
    recorded = rng.integers(1, 9, S).astype(np.int32)
    new = np.where((ctx >= 0) & (ctx <= 40), np.minimum(ctx, 16), 0).astype(np.int32)
    room = [torch.full((S + 2,), -9, dtype=torch.int32, device=cuda_device) for _ in range(2)]
    for t, x in zip(room, (ctx, recorded)):
        t[1:-1] = torch.as_tensor(x)
    given = torch.as_tensor(new, device=cuda_device)
    pa_evict_commit(room[0][1:-1], room[1][1:-1], given)
    torch.cuda.synchronize()
    unusable = (new == 0) & (ctx != 0)
    for t, x in zip(room, (ctx, recorded)):
        want = np.concatenate([[-9], np.where(unusable, x, new), [-9]])
        assert np.array_equal(t.cpu().numpy(), want)
    assert np.array_equal(given.cpu().numpy(), new)
