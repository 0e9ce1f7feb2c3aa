"""pa_decode_weights against attention and its weights in 64 bits."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_444_b200 import (PagedAttentionError, WeightsWorkspace, pa_check_error,
                                     pa_decode, pa_decode_weights, workloads)
from parity_helpers import grow_logits, poison_past_context
from weights_reference import HALF, attend, out_bound

pytestmark = pytest.mark.gpu
BASE = workloads.CONFIGS["gqa_llama3_8b"]


def _batch(dev, ctx, heads, kv_heads, dim, dtype, seed):
    blocks = sum(-(-c // 16) for c in ctx) + 2
    return workloads.make_batch(BASE.scaled(
        name="w", num_seqs=len(ctx), num_heads=heads, num_kv_heads=kv_heads, head_dim=dim,
        dtype=dtype, num_blocks=blocks, ctx=("fixed", tuple(ctx)), seed=seed), dev)


def _call(b, weights, new_tokens=1, scale=None, ws=None, stream=None, out=None):
    out = torch.full_like(b.query, float("nan")) if out is None else out
    ws = ws or WeightsWorkspace.for_call(b.query, b.key_cache, b.block_tables)
    pa_decode_weights(out, weights, ws, b.query, b.key_cache, b.value_cache, b.block_tables,
                      b.context_lens, b.cfg.scale if scale is None else scale, new_tokens, stream)
    return out


def _check(b, before, after, out, new_tokens, scale):
    cfg, G = b.cfg, b.cfg.group_size
    p_half = 2.0 ** -16 if cfg.dtype == "bf16" else 2.0 ** -11
    for s, n in enumerate(b.context_lens.tolist()):
        if n == 0:
            assert (out[s] == 0).all()
            assert torch.equal(after[s].view(torch.int32), before[s].view(torch.int32))
            continue
        at = torch.arange(n, device=out.device)
        blk, row = b.block_tables[s, at // 16].long(), at % 16
        for kv in range(cfg.num_kv_heads):
            k, v = b.key_cache[blk, row, kv], b.value_cache[blk, row, kv]
            q = b.query[s, kv * G:(kv + 1) * G]
            p, o, _, rel, pv = attend(q, k, v, scale)
            err = (out[s, kv * G:(kv + 1) * G].double() - o).abs()
            lim = out_bound(o, pv, rel, n, float(v.double().abs().max()), out.dtype, p_half)
            assert (err <= lim).all(), (s, kv, float((err / lim).max()))
            fresh = max(0, n - new_tokens)
            old = before[s, kv, :n].double().clone()
            old[fresh:] = 0
            want = old + p.sum(0)
            err = (after[s, kv, :n].double() - want).abs()
            lim = (p * rel[:, None]).sum(0) + (G + 2) * 2.0 ** -24 * want.abs() + 1e-37
            assert (err <= lim).all(), (s, kv, float((err / lim).max()))
        assert torch.equal(after[s, :, n:].view(torch.int32), before[s, :, n:].view(torch.int32))


CASES = {
    # name: (contexts, heads, KV heads, head_dim, dtype, new tokens, weight columns over the longest)
    "one_token": ((1,), 1, 1, 64, "f16", 1, 0),
    "tiny": ((1, 9, 16, 37), 4, 4, 64, "f16", 1, 3),
    "empty_between": ((0, 17, 0, 33), 8, 2, 128, "bf16", 1, 1),
    "partition_edges": ((511, 512, 513, 1023, 1025), 8, 2, 128, "bf16", 1, 7),
    "small_partition_edges": ((127, 128, 129, 255, 257, 640), 8, 2, 128, "bf16", 1, 7),
    "small_partitions_group16": ((1281, 100, 256, 0), 16, 1, 64, "f16", 3, 0),
    "group3": ((45, 700), 12, 4, 128, "f16", 1, 0),
    "group2_bf16_d64": ((130, 1), 4, 2, 64, "bf16", 1, 5),
    "group8": ((600, 31), 16, 2, 128, "f16", 2, 0),
    "group9": ((64, 530), 9, 1, 128, "bf16", 1, 0),
    "group12_d64": ((300,), 12, 1, 64, "f16", 1, 2),
    "group16": ((515, 18), 32, 2, 128, "bf16", 1, 0),
    "mha": ((200, 77), 8, 8, 128, "f16", 1, 0),
    "nothing_new": ((100, 20), 8, 2, 128, "bf16", 0, 0),
    "all_new": ((100, 20), 8, 2, 128, "bf16", 1000, 0),
    "long": ((9000, 4097), 8, 2, 128, "bf16", 1, 11),
    "long_mha_d64": ((5001,), 2, 2, 64, "f16", 16, 0),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_the_definition(name, cuda_device):
    ctx, H, Hk, D, dtype, new, extra = CASES[name]
    b = _batch(cuda_device, ctx, H, Hk, D, dtype, 900 + len(name))
    poison_past_context(b)           # rows and weights past a context are never used
    weights = torch.rand((len(ctx), Hk, max(ctx) + extra), device=cuda_device)
    for s, n in enumerate(ctx):
        weights[s, :, max(0, n - new):] = float("nan")
    before = weights.clone()
    out = _call(b, weights, new)
    torch.cuda.synchronize()
    pa_check_error()
    _check(b, before, weights, out, new, b.cfg.scale)


@pytest.mark.parametrize("S,H,Hk,D,dtype", [(120, 16, 8, 128, "bf16"), (120, 128, 8, 64, "f16"),
                                            (300, 4, 4, 128, "f16"), (230, 20, 4, 64, "bf16")])
def test_batches_that_take_a_cta_a_context(S, H, Hk, D, dtype, cuda_device):
    """Enough contexts for two waves of CTAs, ranked by length (up to 256 sequences)
    or not: mostly short ones, empty ones and some of several id windows."""
    rng = np.random.default_rng(S)
    ctx = rng.integers(0, 60, S)
    ctx[[3, S // 2, S - 1]] = (2200, 1777, 2049)
    b = _batch(cuda_device, [int(c) for c in ctx], H, Hk, D, dtype, 960 + S)
    poison_past_context(b)
    weights = torch.rand((S, Hk, 2300), device=cuda_device)
    before = weights.clone()
    out = _call(b, weights)
    torch.cuda.synchronize()
    pa_check_error()
    _check(b, before, weights, out, 1, b.cfg.scale)


@pytest.mark.parametrize("dtype,heads", [("bf16", 8), ("f16", 8), ("bf16", 20)])
def test_climbing_logits(dtype, heads, cuda_device):
    """Row maxima that outgrow the reference several times within a partition."""
    b = _batch(cuda_device, (1500, 300), heads, 2, 128, dtype, 931)
    grow_logits(b)
    weights = torch.zeros((2, 2, 1500), device=cuda_device)
    before = weights.clone()
    out = _call(b, weights)
    torch.cuda.synchronize()
    pa_check_error()
    _check(b, before, weights, out, 1, b.cfg.scale)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_other_scales(scale, cuda_device):
    b = _batch(cuda_device, (700, 33), 8, 2, 64, "bf16", 932)
    weights = torch.zeros((2, 2, 700), device=cuda_device)
    before = weights.clone()
    out = _call(b, weights, scale=scale)
    torch.cuda.synchronize()
    _check(b, before, weights, out, 1, scale)


def test_steps_add_up_to_the_number_of_heads(cuda_device):
    """Three steps over one cache: each adds the group's heads' weight of 1 to every KV head;
    the output is that of pa_decode up to the rounding of P."""
    b = _batch(cuda_device, (777, 1200, 5), 32, 8, 128, "f16", 933)
    ws = WeightsWorkspace.for_call(b.query, b.key_cache, b.block_tables)
    weights = torch.zeros((3, 8, 1200), device=cuda_device)
    out = torch.empty_like(b.query)
    for _ in range(3):
        _call(b, weights, 0, ws=ws, out=out)
    torch.cuda.synchronize()
    total = weights.double().sum(-1)
    # each p is off by rel < 2^-10 at these sizes (module bound), in sum by its mean
    assert (total - 12).abs().max() < 12 * 2.0 ** -10
    plain = torch.empty_like(out)
    pa_decode(plain, b.query, b.key_cache, b.value_cache, b.block_tables, b.context_lens,
              b.cfg.scale)
    assert (plain.float() - out.float()).abs().max() < 2e-3
    pa_check_error()


def test_nan_and_infinite_values_stay_with_their_own_sequence(cuda_device):
    b = _batch(cuda_device, (100, 100, 100), 4, 2, 64, "bf16", 934)
    k_nan, v_inf = int(b.block_tables[0, 2]), int(b.block_tables[1, 3])
    b.key_cache[k_nan, 3, 0] = float("nan")
    b.value_cache[v_inf, 1, 1, 5] = float("inf")
    weights = torch.zeros((3, 2, 100), device=cuda_device)
    before = weights.clone()
    out = _call(b, weights)
    torch.cuda.synchronize()
    assert out[0, :2].isnan().all() and weights[0, 0].isnan().all()
    assert out[0, 2:].isfinite().all() and weights[0, 1].isfinite().all()
    # (bf16 P enters as a hi + lo pair, and lo may be 0 or negative: inf or NaN, as pa_decode)
    assert not out[1, 2:, 5].isfinite().any() and weights[1].isfinite().all()
    rest = out[1].clone()
    rest[2:, 5] = 0
    assert rest.isfinite().all()
    b.context_lens[:2] = 0            # check the third alone
    before[:2], weights[:2], out[:2] = 0, 0, 0
    _check(b, before, weights, out, 1, b.cfg.scale)


def test_reports_bad_lengths_and_blocks(cuda_device):
    b = _batch(cuda_device, (40, 60, 20), 4, 2, 64, "f16", 935)
    weights = torch.full((3, 2, 50), 0.5, device=cuda_device)      # 60 does not fit
    before = weights.clone()
    out = _call(b, weights)
    with pytest.raises(PagedAttentionError, match="context_len, index 1"):
        pa_check_error()
    assert torch.equal(weights[1], before[1])
    plain = torch.empty_like(out)
    pa_decode(plain, b.query, b.key_cache, b.value_cache, b.block_tables, b.context_lens,
              b.cfg.scale)
    assert (plain.float() - out.float()).abs().max() < 2e-3
    wide = torch.zeros((3, 2, 64), device=cuda_device)
    b.block_tables[2, 1] = 1 << 20
    _call(b, wide)
    with pytest.raises(PagedAttentionError, match="block_id, index 9"):
        pa_check_error()
    assert wide.isfinite().all()
    pa_check_error()


def test_graph_and_another_stream(cuda_device):
    b = _batch(cuda_device, (300, 40), 8, 2, 128, "bf16", 936)
    ws = WeightsWorkspace.for_call(b.query, b.key_cache, b.block_tables)
    weights = torch.zeros((2, 2, 320), device=cuda_device)
    out = torch.empty_like(b.query)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _call(b, weights, ws=ws, out=out, stream=side)
    side.synchronize()
    _check(b, torch.zeros_like(weights), weights, out, 1, b.cfg.scale)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(b, weights, ws=ws, out=out)
    for seed in (1, 2):
        b.query.normal_(generator=torch.Generator(device=cuda_device).manual_seed(seed))
        before = weights.clone()
        graph.replay()
        torch.cuda.synchronize()
        _check(b, before, weights, out, 1, b.cfg.scale)
    pa_check_error()


def test_workspace_too_small_is_refused(cuda_device):
    b = _batch(cuda_device, (300, 40), 8, 2, 128, "bf16", 937)
    weights = torch.zeros((2, 2, 320), device=cuda_device)
    small = WeightsWorkspace(1, 8, 128, b.block_tables.shape[1], cuda_device)
    with pytest.raises(PagedAttentionError, match="PA_ERR_SHAPE"):
        _call(b, weights, ws=small)
    assert (weights == 0).all()
    with pytest.raises(ValueError):
        _call(b, weights.double())
    with pytest.raises(ValueError):
        _call(b, weights[:, :1])
    with pytest.raises(PagedAttentionError, match="PA_ERR_SHAPE"):
        _call(b, weights, new_tokens=-1)
    assert math.isfinite(float(weights.sum()))


@pytest.mark.parametrize("n", [40, 1500], ids=["one_cta", "split"])
def test_logits_that_are_all_minus_infinity(n, cuda_device):
    """A product beyond 32 bits: out 0 and nothing added, as for an empty context."""
    b = _batch(cuda_device, (n, 30), 4, 2, 64, "bf16", 938)
    b.query[0] = 0
    b.query[0, :, 0] = 3e38
    own = b.block_tables[0, :-(-n // 16)].long()
    b.key_cache[own] = 0
    b.key_cache[own, :, :, 0] = -3e38
    weights = torch.full((2, 2, n), 0.25, device=cuda_device)
    before = weights.clone()
    out = _call(b, weights, new_tokens=0)
    torch.cuda.synchronize()
    pa_check_error()
    assert (out[0] == 0).all() and torch.equal(weights[0], before[0])
    b.context_lens[0] = 0             # check the other sequence alone
    _check(b, before, weights, out, 0, b.cfg.scale)


def test_offsets_beyond_32_bits(cuda_device):
    """Logits of 50 x 64 heads over tables of 700000 tokens, 2.2e9 in all, and as many weights."""
    ctx = (5,) * 48 + (700_000, 600_001)
    b = _batch(cuda_device, ctx, 64, 4, 64, "bf16", 939)
    weights = torch.full((50, 4, 11_000_000), 0.5, device=cuda_device)
    before = weights[:, :, :700_100].clone()
    out = _call(b, weights)
    torch.cuda.synchronize()
    pa_check_error()
    assert (weights[:, :, 700_100:] == 0.5).all()
    _check(b, before, weights[:, :, :700_100], out, 1, b.cfg.scale)


def test_offsets_beyond_32_bits_with_a_cta_a_context(cuda_device):
    """Logits of 1100 x 64 heads over tables of 32768 tokens, 2.3e9 in all."""
    ctx = (3, 40) * 549 + (32_768, 30_001)
    b = _batch(cuda_device, ctx, 64, 4, 64, "f16", 940)
    weights = torch.zeros((1100, 4, 32_768), device=cuda_device)
    before = weights.clone()
    out = _call(b, weights)
    torch.cuda.synchronize()
    pa_check_error()
    b.context_lens[2:1096] = 0        # check the first and the last ones
    out[2:1096], weights[2:1096] = 0, 0
    _check(b, before, weights, out, 1, b.cfg.scale)


def test_one_workspace_for_batches_of_many_sizes(cuda_device):
    """That of the largest batch, whose partitions are the longest ones."""
    big = _batch(cuda_device, (600,) * 230, 8, 2, 64, "f16", 941)
    ws = WeightsWorkspace.for_call(big.query, big.key_cache, big.block_tables)
    for ctx in ((600,) * 230, (600, 590) * 50, (600, 1, 530), (40, 5)):
        b = _batch(cuda_device, ctx, 8, 2, 64, "f16", 942)
        weights = torch.zeros((len(ctx), 2, 600), device=cuda_device)
        before = weights.clone()
        out = _call(b, weights, ws=ws)
        torch.cuda.synchronize()
        pa_check_error()
        _check(b, before, weights, out, 1, b.cfg.scale)


@pytest.mark.parametrize("n,heads,kv_heads", [(500, 4, 2), (500, 12, 1), (3000, 8, 2), (3000, 9, 1)],
                         ids=["one_cta", "one_cta_wide", "split", "split_wide"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_small_weights_beside_a_large_one(dtype, n, heads, kv_heads, cuda_device):
    """One key takes nearly all of the weight and has no value; the others, at 2^-25.7 to
    2^-26.4 of it, make the output.  Where a warp has both, its fp16 P is below its normal
    numbers: an error of 2^-25 each, against a sum of at least 2^7 (P is held 2^7 up), is 2^-32
    of a value.  It has at most a quarter of 512 tokens."""
    b = _batch(cuda_device, (n, 33), heads, kv_heads, 64, dtype, 943)
    b.query.zero_()
    b.query[..., 0] = 8
    b.key_cache.zero_()
    own = b.block_tables[0, :-(-n // 16)].long()
    step = torch.arange(own.numel() * 16, device=cuda_device).view(-1, 16, 1)
    b.key_cache[own, :, :, 0] = (-9.8125 - 0.25 * (step % 3)).to(b.key_cache.dtype).expand(
        -1, -1, kv_heads)
    b.key_cache[own[0], 0, :, 0] = 8
    b.value_cache.copy_(500 + 500 * torch.rand(b.value_cache.shape, device=cuda_device))
    b.value_cache[own[0], 0] = 0
    weights = torch.zeros((2, kv_heads, n), device=cuda_device)
    before = weights.clone()
    out = _call(b, weights, scale=0.125)
    torch.cuda.synchronize()
    pa_check_error()
    _check(b, before, weights, out, 1, 0.125)
    at, G = torch.arange(n, device=cuda_device), heads // kv_heads
    for kv in range(kv_heads):
        k, v = (c[own[at // 16], at % 16, kv] for c in (b.key_cache, b.value_cache))
        _, o, _, rel, pv = attend(b.query[0, kv * G:(kv + 1) * G], k, v, 0.125)
        half, p_half = HALF[out.dtype], 2.0 ** -16 if dtype == "bf16" else 2.0 ** -11
        lim = (half * o.abs() + (p_half + 2 * rel[:, None] + n * 2.0 ** -23) * pv +
               (128 * 2.0 ** -32 * 1000 + 2.0 ** -25) * (dtype == "f16")) * (1 + half)
        err = (out[0, kv * G:(kv + 1) * G].double() - o).abs()
        assert (err <= lim).all(), (kv, float((err / lim).max()))


def _split_form(rows, cap, group):
    """Tokens of a partition and of a second-pass CTA, as the launch picks them for `rows`
    (sequence, KV head) pairs and tables of `cap` tokens (444: three CTAs an SM)."""
    part, run = 512, 4096
    while part > 128 and rows * -(-cap // part) < 444:
        part //= 2
    while run > 256 and (run * group > 16384 or rows * -(-cap // run) < 444):
        run //= 2
    return part, run


SPLITS = {
    # name: (contexts, heads, KV heads, head_dim, partition, run)
    "parts_512": ((511, 512, 513, 1023, 1024, 1025) + (5,) * 24, 32, 8, 128, 512, 1024),
    "parts_512_mha": ((512, 1025, 513, 1, 0, 1024) + (3,) * 14, 16, 16, 128, 512, 1024),
    "parts_512_group16_d64": ((511, 512, 513, 1025) + (7,) * 226, 16, 1, 64, 512, 1024),
    "runs_4096": ((4095, 4096, 4097, 8192, 8193, 28672, 512, 1), 32, 8, 128, 512, 4096),
    "runs_2048_group8": ((2047, 2048, 2049, 4096, 28001, 513, 0, 1), 64, 8, 128, 512, 2048),
    "runs_1024_group16": ((1023, 1024, 1025, 3073, 30000) + (17,) * 11, 64, 4, 128, 512, 1024),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name", SPLITS)
def test_edges_of_the_longest_partitions_and_runs(name, dtype, cuda_device):
    """The two-launch form as large batches take it: contexts at the ends of partitions of 512
    tokens and of second-pass runs."""
    ctx, H, Hk, D, part, run = SPLITS[name]
    b = _batch(cuda_device, ctx, H, Hk, D, dtype, 970 + len(name))
    rows, cap = len(ctx) * Hk, b.block_tables.shape[1] * 16
    assert _split_form(rows, cap, H // Hk) == (part, run) and cap > 512
    assert rows < 6 * 148 or cap <= 1536          # (else a CTA takes a context)
    poison_past_context(b)
    weights = torch.rand((len(ctx), Hk, max(ctx) + 3), device=cuda_device)
    before = weights.clone()
    out = _call(b, weights)
    torch.cuda.synchronize()
    pa_check_error()
    _check(b, before, weights, out, 1, b.cfg.scale)
