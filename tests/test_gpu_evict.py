"""pa_evict_select and pa_evict_compact against a plain restatement on the host:
whole numbers and moved bits, so every comparison is for equality."""
import numpy as np
import pytest
import torch

import evict_reference as ref
from paged_kv_cache_444_b200 import (PagedAttentionError, pa_check_error, pa_evict_compact,
                                     pa_evict_select)

pytestmark = pytest.mark.gpu


def _i32(x, dev):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=dev)


class Batch:
    """Random weights and positions of a batch; `recorded` slots a sequence
    were placed by an earlier eviction, the others follow in order."""

    def __init__(self, dev, ctx, Hk, budget, seed, recorded=None, W=None, weights=None, age=7):
        rng = np.random.default_rng(seed)
        S = len(ctx)
        self.W = W or max(max(ctx), 1)
        self.budget, self.Hk, self.dev = budget, Hk, dev
        self.ctx = np.array(ctx, dtype=np.int32)
        self.recorded = np.array(recorded if recorded is not None else [0] * S, dtype=np.int32)
        self.length = np.where(self.recorded > 0, self.ctx * age, self.ctx).astype(np.int32)
        self.weights = (np.exp(2 * rng.standard_normal((S, Hk, self.W))).astype(np.float32)
                        if weights is None else weights(rng, (S, Hk, self.W)))
        self.positions = rng.integers(-9, 9, (S, Hk, self.W)).astype(np.int32)  # unread garbage
        for s in range(S):
            r = int(self.recorded[s])
            for h in range(Hk):
                first = int(self.length[s]) - (int(self.ctx[s]) - r)
                self.positions[s, h, :r] = rng.permutation(first)[:r]
        self.t = {k: torch.as_tensor(getattr(self, k), device=dev) for k in
                  ("weights", "positions", "ctx", "recorded", "length")}
        self.source = torch.full((S, Hk, budget), -7, dtype=torch.int32, device=dev)
        self.new_lens = torch.full((S,), -7, dtype=torch.int32, device=dev)

    def select(self, sink, recent, stream=None):
        pa_evict_select(self.source, self.new_lens, self.t["weights"], self.t["positions"],
                        self.t["ctx"], self.t["recorded"], self.t["length"], sink, recent, stream)

    def want(self, sink, recent):
        return ref.select(self.weights, self.positions, self.recorded, self.length, self.ctx,
                          self.budget, sink, recent)

    def check_select(self, sink, recent):
        self.select(sink, recent)
        torch.cuda.synchronize()
        pa_check_error()
        source, new = self.want(sink, recent)
        assert np.array_equal(self.new_lens.cpu().numpy(), new)
        got = self.source.cpu().numpy()
        bad = np.argwhere(got != source)
        assert bad.size == 0, (bad[:4], got[tuple(bad[0])], source[tuple(bad[0])])


def _ties(rng, shape):       # few values, both zeros among them
    return rng.choice(np.array([0.0, -0.0, 0.25, 0.5], dtype=np.float32), shape)


def _equal(rng, shape):
    return np.full(shape, 0.125, dtype=np.float32)


def _odd(rng, shape):        # NaN, infinities, denormals, negatives
    w = rng.standard_normal(shape).astype(np.float32)
    pick = rng.integers(0, 8, shape)
    w[pick == 0] = np.nan
    w[pick == 1] = np.inf
    w[pick == 2] = -np.inf
    w[pick == 3] = 1e-42
    return w


SELECT = {
    # name: (contexts, KV heads, budget, sink, recent, options)
    "one_token": ((1,), 1, 1, 0, 0, {}),
    "two_of_three": ((3,), 2, 2, 1, 1, {}),
    "empty_and_short": ((0, 1, 5, 6, 7), 3, 6, 1, 2, {}),
    "one_over": ((33, 34, 65), 2, 32, 4, 8, {}),
    "all_held": ((40, 50), 2, 32, 12, 20, {}),
    "nothing_held": ((1000, 31, 999), 2, 100, 0, 0, {}),
    "odd_width": ((777, 1025, 1024), 3, 333, 4, 50, dict(W=1111)),
    "steady": ((130, 147, 129), 4, 128, 4, 30, dict(recorded=(128, 128, 128))),
    "steady_mixed": ((130, 100, 300), 2, 128, 2, 16, dict(recorded=(128, 0, 128))),
    "budget_over_width": ((50, 60), 2, 100, 4, 8, {}),
    "ties": ((500, 2000), 2, 200, 3, 10, dict(weights=_ties)),
    "equal": ((700, 1300), 2, 512, 0, 5, dict(weights=_equal)),
    "odd_values": ((900, 1500), 2, 300, 4, 10, dict(weights=_odd)),
    "mostly_nan": ((400,), 1, 390, 0, 0, dict(weights=_odd)),
    "long": ((20000, 16384, 9), 2, 3000, 4, 100, {}),
    "cluster_ties": ((40000,), 2, 25000, 4, 100, dict(weights=_ties)),
    "cluster_of_eight": ((131072, 70001), 1, 4096, 4, 512, {}),
    "cluster_equal": ((100001,), 1, 60000, 1, 7, dict(weights=_equal)),
    "wide_table": ((300, 200), 2, 100, 4, 10, dict(W=524288)),
}


@pytest.mark.parametrize("name", SELECT)
def test_select_matches_the_plain_form(name, cuda_device):
    ctx, Hk, budget, sink, recent, kw = SELECT[name]
    Batch(cuda_device, ctx, Hk, budget, 500 + len(name), **kw).check_select(sink, recent)


@pytest.mark.parametrize("weights", [None, _ties, _odd], ids=["random", "ties", "odd"])
@pytest.mark.parametrize("n,budget,recorded", [(1100, 1000, 1000), (4113, 4096, 4096),
                                               (9000, 5000, 0), (12000, 3500, 3500)])
def test_select_with_more_rows_than_ctas_at_once(n, budget, recorded, weights, cuda_device):
    """300 rows: one CTA a row, its keys in registers up to 9216 slots."""
    S = 300
    b = Batch(cuda_device, (n,) * S, 1, budget, 97, weights=weights,
              recorded=(recorded,) * S if recorded else None)
    b.select(4, 60)
    torch.cuda.synchronize()
    pa_check_error()
    got = b.source.cpu().numpy()
    for s in (0, 101, 202, 299):
        want = ref.select_row(b.weights[s, 0], b.positions[s, 0], recorded, int(b.length[s]), n,
                              budget, 4, 60)
        assert np.array_equal(got[s, 0], want), s


def test_select_where_keys_do_not_fit_shared_memory(cuda_device):
    """The longest context the call takes: a CTA's run of 65536 slots is read
    again after its first digit.  numpy's stable sort stands in for the slow loop."""
    n, B, sink, recent = 524288, 200000, 4, 1000
    b = Batch(cuda_device, (n,), 1, B, 91)
    b.select(sink, recent)
    torch.cuda.synchronize()
    pa_check_error()
    w = b.weights[0, 0].astype(np.float64)
    w[:sink] = np.inf
    w[n - recent:] = np.inf
    kept = np.zeros(n, bool)
    kept[np.argsort(-w, kind="stable")[:B]] = True
    want = np.arange(B)
    want[~kept[:B]] = B + np.flatnonzero(kept[B:])
    assert np.array_equal(b.source[0, 0].cpu().numpy(), want)


@pytest.mark.parametrize("budget", [12000, 16384])
def test_select_many_rows_of_a_wide_table(budget, cuda_device):
    """More rows than clusters for each fit the device, and tables so wide that one CTA's
    flags and list would not fit its shared memory."""
    S, W, n = 160, 1 << 19, 30000
    g = torch.Generator(device=cuda_device).manual_seed(96)
    weights = torch.rand((S, 1, W), generator=g, device=cuda_device)
    positions = torch.zeros((S, 1, W), dtype=torch.int32, device=cuda_device)
    lens = torch.full((S,), n, dtype=torch.int32, device=cuda_device)
    zeros, new = torch.zeros_like(lens), torch.empty_like(lens)
    source = torch.full((S, 1, budget), -7, dtype=torch.int32, device=cuda_device)
    pa_evict_select(source, new, weights, positions, lens, zeros, lens.clone(), 4, 100)
    torch.cuda.synchronize()
    pa_check_error()
    assert (new == budget).all()
    for s in (0, 77, 159):
        w = weights[s, 0, :n].cpu().numpy().astype(np.float64)
        w[:4] = w[n - 100:] = np.inf
        kept = np.zeros(n, bool)
        kept[np.argsort(-w, kind="stable")[:budget]] = True
        want = np.arange(budget)
        want[~kept[:budget]] = budget + np.flatnonzero(kept[budget:])
        assert np.array_equal(source[s, 0].cpu().numpy(), want)


def test_select_reports_a_bad_context_length(cuda_device):
    b = Batch(cuda_device, (50, 60, 20), 2, 16, 92)
    b.t["ctx"] = _i32([50, 61, 20], cuda_device)      # past max_tokens
    b.select(1, 4)
    with pytest.raises(PagedAttentionError, match="context_len, index 1"):
        pa_check_error()
    pa_check_error()                                  # cleared
    source, new = b.want(1, 4)
    assert np.array_equal(b.new_lens.cpu().numpy(), [16, 0, 16])
    got = b.source.cpu().numpy()
    assert np.array_equal(got[[0, 2]], source[[0, 2]]) and (got[1] == -1).all()


def _caches(dev, b, D, dtype, bs, seed, spare=3):
    """Caches of random bits and tables of distinct blocks, -1 past each end."""
    rng = np.random.default_rng(seed)
    need = [-(-int(c) // bs) for c in b.ctx]
    width = max(1, *need)
    perm = rng.permutation(sum(need) + spare).astype(np.int32)
    tables, at = np.full((len(need), width), -1, dtype=np.int32), 0
    for s, m in enumerate(need):
        tables[s, :m] = perm[at:at + m]
        at += m
    kind = np.uint8 if dtype == torch.uint8 else np.uint16
    shape = (sum(need) + spare, bs, b.Hk, D)
    kc, vc = (rng.integers(0, np.iinfo(kind).max, shape, endpoint=True).astype(kind)
              for _ in range(2))
    to = lambda x: torch.as_tensor(x.view(np.int16) if kind == np.uint16 else x,
                                   device=dev).view(dtype)
    return kc, vc, tables, to(kc), to(vc)


def _bits(t):
    t = t.cpu()
    return t.numpy() if t.dtype == torch.uint8 else t.view(torch.int16).numpy().view(np.uint16)


COMPACT = {
    # name: (select case, head_dim, dtype, block size)
    "tiny_f16": ("two_of_three", 64, torch.float16, 16),
    "empty_bf16": ("empty_and_short", 128, torch.bfloat16, 16),
    "one_over_fp8": ("one_over", 128, torch.uint8, 16),
    "nothing_held_bf16": ("nothing_held", 128, torch.bfloat16, 16),
    "odd_width_d8": ("odd_width", 8, torch.float16, 16),
    "steady_bf16": ("steady", 128, torch.bfloat16, 16),
    "steady_mixed_f16": ("steady_mixed", 64, torch.float16, 16),
    "budget_over_width": ("budget_over_width", 128, torch.bfloat16, 16),
    "block_of_five": ("one_over", 16, torch.uint8, 5),
    "long_bf16": ("long", 64, torch.bfloat16, 16),
}


@pytest.mark.parametrize("name", COMPACT)
def test_compact_moves_what_select_kept(name, cuda_device):
    case, D, dtype, bs = COMPACT[name]
    ctx, Hk, budget, sink, recent, kw = SELECT[case]
    b = Batch(cuda_device, ctx, Hk, budget, 700 + len(name), **kw)
    kc, vc, tables, kd, vd = _caches(cuda_device, b, D, dtype, bs, 701)
    b.select(sink, recent)
    source, new = b.want(sink, recent)
    want = ref.compact(kc, vc, b.weights, b.positions, source, new, tables, b.ctx, b.recorded,
                       b.length)
    td = torch.as_tensor(tables, device=cuda_device)
    for again in range(2):     # repeating the call changes nothing
        pa_evict_compact(kd, vd, b.t["weights"], b.t["positions"], b.source, b.new_lens, td,
                         b.t["ctx"], b.t["recorded"], b.t["length"])
        torch.cuda.synchronize()
        pa_check_error()
        assert np.array_equal(_bits(kd), want[0]) and np.array_equal(_bits(vd), want[1])
        assert np.array_equal(b.t["weights"].cpu().numpy(), want[2])
        assert np.array_equal(b.t["positions"].cpu().numpy(), want[3])


def test_compact_leaves_out_bad_sources_and_blocks(cuda_device):
    """A source out of range and a block id out of range are reported, their
    moves left out; a new length that cannot be is reported, its sequence left."""
    b = Batch(cuda_device, (40, 40, 40), 1, 20, 93, weights=_equal)
    kc, vc, tables, kd, vd = _caches(cuda_device, b, 64, torch.float16, 16, 94)
    b.select(0, 5)                                   # slots 15..19 <- 35..39
    source, new = b.want(0, 5)
    assert (source[0, 0, 15:] == np.arange(35, 40)).all()

    def run(src, lens, tab):
        w, p = b.t["weights"].clone(), b.t["positions"].clone()
        k, v = kd.clone(), vd.clone()
        pa_evict_compact(k, v, w, p, _i32(src, cuda_device), _i32(lens, cuda_device),
                         torch.as_tensor(tab, device=cuda_device), b.t["ctx"], b.t["recorded"],
                         b.t["length"])
        return k, v

    bad = source.copy()
    bad[1, 0, 17] = 40                               # at the context's end
    good = source.copy()
    good[1, 0, 17] = 17
    k, v = run(bad, new, tables)
    with pytest.raises(PagedAttentionError, match="source, index 37"):
        pa_check_error()
    want = ref.compact(kc, vc, b.weights, b.positions, good, new, tables, b.ctx, b.recorded,
                       b.length)
    assert np.array_equal(_bits(k), want[0]) and np.array_equal(_bits(v), want[1])

    bad[1, 0, 17] = 3                                # below the new length, not itself
    k, _ = run(bad, new, tables)
    with pytest.raises(PagedAttentionError, match="source, index 37"):
        pa_check_error()
    assert np.array_equal(_bits(k), want[0])

    broken = tables.copy()
    broken[2, 2] = kc.shape[0]                       # slots 32.. of sequence 2
    stay = source.copy()
    stay[2, 0, 15:] = np.arange(15, 20)
    k, v = run(source, new, broken)
    with pytest.raises(PagedAttentionError, match="block_id, index 8"):
        pa_check_error()
    want = ref.compact(kc, vc, b.weights, b.positions, stay, new, tables, b.ctx, b.recorded,
                       b.length)
    assert np.array_equal(_bits(k), want[0]) and np.array_equal(_bits(v), want[1])

    k, v = run(source, [20, 21, 20], tables)         # more than the budget
    with pytest.raises(PagedAttentionError, match="context_len, index 1"):
        pa_check_error()
    stay = source.copy()
    stay[1, 0, 15:] = np.arange(15, 20)
    want = ref.compact(kc, vc, b.weights, b.positions, stay, new, tables, b.ctx, b.recorded,
                       b.length)
    assert np.array_equal(_bits(k), want[0])
    pa_check_error()


def test_select_on_another_stream_and_in_a_graph(cuda_device):
    """The call goes to the stream it is given, and replays read the buffers' new contents."""
    b = Batch(cuda_device, (600, 90), 2, 64, 95)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    b.select(2, 8, stream=other)
    other.synchronize()
    assert np.array_equal(b.source.cpu().numpy(), b.want(2, 8)[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.select(2, 8)
    for seed in (1, 2):
        b.weights = np.random.default_rng(seed).random(b.weights.shape, dtype=np.float32)
        b.t["weights"].copy_(torch.as_tensor(b.weights))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(b.source.cpu().numpy(), b.want(2, 8)[0])
    pa_check_error()


def test_offsets_beyond_32_bits(cuda_device):
    """Weights of 520 x 8 rows of 2^19 columns and caches of 2.6e9 elements."""
    S, Hk, W, B, D = 520, 8, 1 << 19, 40, 64
    dev, g = cuda_device, torch.Generator(device=cuda_device).manual_seed(98)
    weights = torch.full((S, Hk, W), 7.0, device=dev)
    weights[:, :, :100] = torch.rand((S, Hk, 100), generator=g, device=dev)
    positions = torch.full((S, Hk, W), -5, dtype=torch.int32, device=dev)
    ctx = torch.full((S,), 97, dtype=torch.int32, device=dev)
    rec, length = torch.zeros_like(ctx), ctx.clone()
    source = torch.full((S, Hk, B), -7, dtype=torch.int32, device=dev)
    new = torch.empty_like(ctx)
    NB = 320_000
    kc = torch.zeros((NB, 16, Hk, D), dtype=torch.float16, device=dev)
    vc = torch.zeros_like(kc)
    tables = torch.arange(S * 7, dtype=torch.int32, device=dev).view(S, 7)
    tables = NB - 1 - tables.flip(0)                  # the last blocks belong to the last rows
    at = tables.long()
    kc[at], vc[at] = (torch.randn((S, 7, 16, Hk, D), generator=g, device=dev).half()
                      for _ in range(2))
    few = [0, 300, S - 2, S - 1]
    w0 = weights[few, :, :97].cpu().numpy()
    k0, v0 = (x[at[few]].cpu().view(torch.int16).numpy().reshape(-1, 16, Hk, D) for x in (kc, vc))
    pa_evict_select(source, new, weights, positions, ctx, rec, length, 2, 5)
    pa_evict_compact(kc, vc, weights, positions, source, new, tables, ctx, rec, length)
    torch.cuda.synchronize()
    pa_check_error()
    p0, lens = np.zeros_like(w0, dtype=np.int32), np.full(4, 97, np.int32)
    want, nw = ref.select(w0, p0, 0 * lens, lens, lens, B, 2, 5)
    assert np.array_equal(source[few].cpu().numpy(), want) and (new == B).all()
    local = np.arange(28, dtype=np.int32).reshape(4, 7)
    k1, v1, w1, p1 = ref.compact(k0, v0, w0, p0, want, nw, local, lens, 0 * lens, lens)
    for got, ours in ((kc, k1), (vc, v1)):
        got = got[at[few]].cpu().view(torch.int16).numpy().reshape(-1, 16, Hk, D)
        assert np.array_equal(got, ours)
    assert np.array_equal(weights[few, :, :97].cpu().numpy(), w1)
    assert np.array_equal(positions[few, :, :B].cpu().numpy(), p1[:, :, :B])
    assert (positions[:, :, B:] == -5).all() and (weights[:, :, 100:] == 7).all()


def _few_numbers(rng, shape):
    """Fewer numbers than the budget, the rest NaN: NaN's key decides."""
    w = np.full(shape, np.nan, np.float32)
    w[rng.random(shape) < 0.2] = 1.5
    return w


@pytest.mark.parametrize("ctx,Hk,budget,recorded", [
    ((45, 333, 31), 2, 20, (0, 250, 0)), ((1101,) * 3, 1, 900, (900,) * 3),
    ((5001, 4977), 1, 3000, None), ((60001, 33), 1, 20000, None),
    ((333,) * 200, 1, 200, None), ((41, 570) * 100, 1, 30, None),
], ids=["tiny", "steady", "registers", "streamed", "one_warp", "one_warp_18"])
def test_select_where_nan_decides(ctx, Hk, budget, recorded, cuda_device):
    b = Batch(cuda_device, ctx, Hk, budget, 99, recorded=recorded, weights=_few_numbers)
    b.check_select(2, 11)


@pytest.mark.parametrize("weights", [None, _ties, _odd, _few_numbers],
                         ids=["random", "ties", "odd", "nan"])
@pytest.mark.parametrize("n,Hk,B", [(131072, 1, 4096), (100001, 2, 30000)])
def test_select_of_few_long_rows(n, Hk, B, weights, cuda_device):
    """Up to 16384 slots a CTA in registers, an SM for each.  A stable sort stands in for the
    slow loop."""
    b = Batch(cuda_device, (n,), Hk, B, 90, weights=weights)
    b.select(4, 50)
    torch.cuda.synchronize()
    pa_check_error()
    for h in range(Hk):
        w = b.weights[0, h].astype(np.float64)
        rank = np.where(np.isnan(w), -np.inf, w)
        lower = np.isnan(w)                       # NaN counts below -inf
        held = np.zeros(n, bool)
        held[:4] = held[n - 50:] = True
        order = np.lexsort((np.arange(n), -rank, lower, ~held))
        kept = np.zeros(n, bool)
        kept[order[:B]] = True
        want = np.arange(B)
        want[~kept[:B]] = B + np.flatnonzero(kept[B:])
        assert np.array_equal(b.source[0, h].cpu().numpy(), want)


@pytest.mark.parametrize("block", [None, 2, 1], ids=["source", "from", "to"])
def test_compact_leaves_a_slot_whole_where_its_move_is_left_out(block, cuda_device):
    """A move that is left out, for its source or for the block id at either end, leaves
    the slot's weight and position beside its own K and V rows; the position is recorded."""
    b = Batch(cuda_device, (40, 40, 40), 2, 20, 87, recorded=(0, 17, 30))
    kc, vc, tables, kd, vd = _caches(cuda_device, b, 64, torch.float16, 16, 88)
    source = np.broadcast_to(np.arange(20, dtype=np.int32), (3, 2, 20)).copy()
    source[:, :, 14:] = np.arange(34, 40)              # slots 14, 15 and 16 .. 19
    new, stay = np.full(3, 20, dtype=np.int32), source.copy()
    given, broken = source.copy(), tables.copy()
    for s in range(3):
        if block is None:
            given[s, 1, 18] = (40, 3, -1)[s]
            stay[s, 1, 18] = 18
        else:
            broken[s, block] = (-1, len(kc), 1 << 30)[s]
            at = slice(14, 20) if block == 2 else slice(16, 20)
            stay[s, :, at] = np.arange(20)[at]
    want = ref.compact(kc, vc, b.weights, b.positions, stay, new, tables, b.ctx, b.recorded,
                       b.length)
    w, p = b.t["weights"], b.t["positions"]
    for again in range(2):
        pa_evict_compact(kd, vd, w, p, _i32(given, cuda_device), _i32(new, cuda_device),
                         _i32(broken, cuda_device), b.t["ctx"], b.t["recorded"], b.t["length"])
        with pytest.raises(PagedAttentionError, match="source" if block is None else "block_id"):
            pa_check_error()
        assert np.array_equal(_bits(kd), want[0]) and np.array_equal(_bits(vd), want[1])
        assert np.array_equal(w.cpu().numpy(), want[2])
        assert np.array_equal(p.cpu().numpy(), want[3])
