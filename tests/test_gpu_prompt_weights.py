"""pa_prompt_weights against the sums of the attention's weights in 64 bits."""
import numpy as np
import pytest
import torch

from paged_kv_cache_444_b200 import (PagedAttentionError, pa_check_error, pa_prompt_attention,
                                     pa_prompt_weights)
from test_gpu_prompt import Prompt, _draw

pytestmark = pytest.mark.gpu


def _lse(p, scale=None):
    """The attention's lse of every row, and the scale."""
    p.run(scale)
    return p.lse, p.scale


def _check(p, weights, lse, window, seqs=None, fill=7.0):
    """Each term exp(z - lse) is off by rel (z and 2^x; lse is an input here), a tile's 128
    terms are added in chains of 32 and the tiles one after another: 2^-24 a step."""
    torch.cuda.synchronize()
    pa_check_error()
    starts, G = p.starts.tolist(), p.H // p.Hk
    for s in range(len(p.lens)) if seqs is None else seqs:
        b, n = starts[s], p.lens[s]
        assert (weights[s, :, n:] == fill).all()
        if n == 0:
            continue
        first = max(0, n - window)
        later = torch.ones((n - first, n), dtype=torch.bool, device=weights.device).triu(first + 1)
        for kv in range(p.Hk):
            k = p.k[b:b + n, kv].double()
            want, lim = torch.zeros(n, device=k.device).double(), 1e-37
            for h in range(kv * G, (kv + 1) * G):
                q = p.q[b + first:b + n, h].double()
                z = (q @ k.T * p.scale).masked_fill(later, -torch.inf)
                x = z - lse[b + first:b + n, h, None].double()
                size = (q.abs() @ k.abs().T * abs(p.scale)).masked_fill(later, 0)
                rel = (p.D * 2.0 ** -23 * size + 4 * 2.0 ** -24 *
                       (z.abs().masked_fill(later, 0) + lse[b + first:b + n, h, None].abs()) +
                       2.0 ** -21)
                want = want + x.exp().sum(0)
                lim = lim + (x.exp() * rel).sum(0)
            steps = 40 + (n - first) * G // 100
            err = (weights[s, kv, :n].double() - want).abs()
            lim = lim + steps * 2.0 ** -24 * want
            assert (err <= lim).all(), (s, kv, float((err / lim).max()))


def _run(p, window, scale=None, extra=0):
    lse, scale = _lse(p, scale)
    weights = torch.full((len(p.lens), p.Hk, max(max(p.lens), 1) + extra), 7.0,
                         device=p.q.device)
    pa_prompt_weights(weights, p.q, p.k, lse, p.starts, scale, window)
    return weights, lse


CASES = {
    # name: (lengths, heads, KV heads, head_dim, dtype, window, options)
    "one_token": ((1,), 1, 1, 64, "f16", 1, {}),
    "tiny": ((1, 9, 16, 37), 4, 4, 64, "f16", 8, dict(trail=3)),
    "last_token": ((300, 17, 513), 8, 2, 128, "bf16", 1, dict(fused=True)),
    "key_edges_mha": ((127, 128, 129, 255, 256, 257), 2, 2, 128, "bf16", 1000, dict(lead=5)),
    "key_edges_gqa4": ((127, 129, 255, 257, 385, 511), 8, 2, 128, "f16", 1000, {}),
    "empty_between": ((0, 50, 0, 70, 0), 8, 2, 64, "bf16", 33, dict(lead=2, trail=9)),
    "group3": ((45, 400, 1), 12, 4, 128, "f16", 300, dict(fused=True)),
    "group5_d64": ((330, 27), 5, 1, 64, "f16", 1000, dict(trail=1)),
    "group9": ((99, 340), 9, 1, 128, "bf16", 64, {}),
    "group16": ((700, 50), 32, 2, 128, "bf16", 100, {}),
    "window_32": ((513, 77, 1210, 640), 8, 2, 128, "bf16", 32, dict(fused=True, trail=11)),
    "whole_gqa8_d64": ((1500, 1100), 8, 1, 64, "f16", 5000, {}),
    "whole_mha": ((1900, 1025), 2, 2, 128, "bf16", 1900, {}),
    "long_whole": ((6000,), 4, 1, 128, "bf16", 6000, {}),
    # few items: clusters of 2, 4 and 8 CTAs, some without a tile of a key block
    "pair_of_ctas": ((200,), 2, 1, 64, "f16", 130, {}),
    "four_ctas": ((777, 5, 300), 4, 1, 128, "bf16", 140, dict(trail=7)),
    "eight_ctas_mqa": ((3000, 1700), 16, 1, 128, "f16", 3000, dict(fused=True)),
    "eight_ctas_group3": ((1000,), 6, 2, 64, "bf16", 1000, {}),
    "eight_ctas_many_items": ((9000,), 16, 1, 64, "f16", 9000, {}),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_the_definition(name, cuda_device):
    lens, H, Hk, D, dtype, window, kw = CASES[name]
    p = Prompt(cuda_device, lens, H, Hk, D, dtype, 60 + len(name), **kw)
    weights, lse = _run(p, window, extra=len(name) % 3)
    _check(p, weights, lse, window)


@pytest.mark.parametrize("lens,H,Hk,seqs", [
    (_draw(1, 256, 40), 4, 2, range(0, 256, 5)),
    (_draw(2, 300, 40), 4, 2, range(0, 300, 7)),
    (_draw(3, 1200, 9), 4, 1, range(0, 1200, 31)),
], ids=["256", "300", "1200"])
def test_many_sequences(lens, H, Hk, seqs, cuda_device):
    p = Prompt(cuda_device, lens, H, Hk, 64, "bf16", 71)
    weights, lse = _run(p, 16)
    _check(p, weights, lse, 16, seqs)
    live = torch.arange(weights.shape[2], device=cuda_device) < torch.tensor(
        lens, device=cuda_device)[:, None, None]
    assert ((weights == 7) == ~live.expand_as(weights)).all()     # every token was written


@pytest.mark.parametrize("scale", [1.0, 0.0, -0.2])
def test_other_scales(scale, cuda_device):
    p = Prompt(cuda_device, (700, 133), 8, 2, 128, "f16", 72)
    weights, lse = _run(p, 700, scale)
    _check(p, weights, lse, 700)


def test_every_token_gives_a_weight_of_one(cuda_device):
    """Over a whole prompt each query row's weights add up to 1: n G a KV head."""
    p = Prompt(cuda_device, (900, 333), 8, 2, 128, "bf16", 73)
    weights, _ = _run(p, 900)
    torch.cuda.synchronize()
    for s, n in enumerate(p.lens):
        total = weights[s, :, :n].double().sum(-1)
        # a row's p are off by 2 rel < 2^-10 at these sizes
        assert (total - 4 * n).abs().max() < 4 * n * 2.0 ** -10


def test_what_is_not_seen_does_not_count(cuda_device):
    """NaN rows of another sequence, of later queries outside the tile's sequence, and of a
    key: a key sums the tokens at or behind it of its own sequence alone."""
    p = Prompt(cuda_device, (150, 90, 260), 8, 2, 128, "bf16", 74)
    lse, scale = _lse(p)
    lse, b = lse.clone(), p.starts.tolist()
    p.q[b[1]:b[2]] = float("nan")              # the next sequence's queries
    p.k[b[1]:b[2]] = float("inf")
    lse[b[1]:b[2]] = float("nan")
    p.q[b[2] + 40] = float("nan")              # an earlier query of sequence 2, keys <= 40
    p.k[b[2] + 200, 1] = float("nan")          # a key of sequence 2
    weights = torch.full((3, 2, 260), 7.0, device=cuda_device)
    pa_prompt_weights(weights, p.q, p.k, lse, p.starts, scale, 260)
    _check(p, weights, lse, 260, seqs=[0])
    assert weights[1, :, :90].isnan().all() and (weights[1, :, 90:] == 7).all()
    assert weights[2, :, :41].isnan().all() and weights[2, 0, 41:].isfinite().all()
    assert weights[2, 1, 200].isnan() and weights[2, 1, 201:].isfinite().all()
    assert weights[2, 1, 41:200].isfinite().all()
    # a row without any finite logit has lse = -inf and gives nothing
    lse[b[0] + 149] = float("-inf")
    p.q[b[0] + 149] = 0
    pa_prompt_weights(weights, p.q, p.k, lse, p.starts, scale, 1)
    torch.cuda.synchronize()
    assert (weights[0, :, :150] == 0).all()


def test_reports_long_sequences_and_bad_bounds(cuda_device):
    p = Prompt(cuda_device, (40, 70, 60), 4, 2, 64, "f16", 75)
    lse, scale = _lse(p)
    weights = torch.full((3, 2, 64), 7.0, device=cuda_device)
    pa_prompt_weights(weights, p.q, p.k, lse, p.starts, scale, 8)
    with pytest.raises(PagedAttentionError, match="context_len, index 1"):
        pa_check_error()
    assert (weights[1] == 7).all()
    _check(p, weights, lse, 8, seqs=[0, 2])
    p.starts[3] = p.T + 1
    pa_prompt_weights(weights, p.q, p.k, lse, p.starts, scale, 8)
    with pytest.raises(PagedAttentionError):
        pa_check_error()
    pa_check_error()


def test_repeats_are_equal_and_graphs_replay(cuda_device):
    p = Prompt(cuda_device, (640, 900), 8, 2, 128, "bf16", 76)
    one, lse = _run(p, 900)
    two = torch.full_like(one, 7.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa_prompt_weights(two, p.q, p.k, lse, p.starts, p.scale, 900, stream=side)
    side.synchronize()
    assert torch.equal(one, two)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):     # both calls, as a program makes them
        pa_prompt_attention(p.out, p.lse, p.q, p.k, p.v, p.starts, p.scale)
        pa_prompt_weights(two, p.q, p.k, p.lse, p.starts, p.scale, 64)
    p.k.normal_()
    two.fill_(7)
    graph.replay()
    _check(p, two, p.lse, 64)


def test_binding_refuses(cuda_device):
    p = Prompt(cuda_device, (20, 30), 8, 2, 64, "f16", 77)
    lse, scale = _lse(p)
    a = dict(weights=torch.zeros((2, 2, 30), device=cuda_device), query=p.q, key=p.k, lse=lse,
             seq_starts=p.starts, scale=scale, window=4)
    for bad in (dict(weights=a["weights"][:1]), dict(weights=a["weights"].half()),
                dict(lse=lse[:, :4]), dict(lse=lse.T), dict(key=p.k.bfloat16()),
                dict(seq_starts=p.starts.long()), dict(lse=lse.cpu())):
        with pytest.raises(ValueError):
            pa_prompt_weights(**{**a, **bad})
    for bad in (dict(window=0), dict(window=-3), dict(scale=float("inf"))):
        with pytest.raises(PagedAttentionError, match="PA_ERR_SHAPE"):
            pa_prompt_weights(**{**a, **bad})
    assert np.isfinite(float(a["weights"].sum()))


def test_offsets_beyond_32_bits(cuda_device):
    """Weights of 40 x 8 rows of 7 million columns, 2.2e9 in all."""
    p = Prompt(cuda_device, tuple(range(1, 41)), 8, 8, 64, "f16", 79)
    weights, lse = _run(p, 100, extra=7_000_000 - 40)
    _check(p, weights, lse, 100, seqs=[0, 38, 39])


@pytest.mark.parametrize("H,Hk", [(6, 2), (5, 1), (13, 1), (8, 2)])
def test_a_key_with_logits_of_minus_infinity_gets_no_weight(H, Hk, cuda_device):
    """exp(-inf - lse) is 0 for it in full tiles too, whose last columns hold no query row
    where the group does not divide 128."""
    p = Prompt(cuda_device, (400, 333), H, Hk, 64, "bf16", 80)
    p.q[:, :, 0] = 1 + p.q[:, :, 0].abs()
    p.k[[7, 150, 407]] = 0
    p.k[[7, 150, 407], :, 0] = -torch.inf
    weights, lse = _run(p, 1000)
    torch.cuda.synchronize()
    pa_check_error()
    assert lse.isfinite()[8:400].all() and lse.isfinite()[408:].all()
    gone = [(0, 7), (0, 150), (1, 7)]
    for s, j in gone:
        assert (weights[s, :, j] == 0).all(), (s, j, weights[s, :, j])
    # the others are what they are when those keys are as far as 16 bits go
    p.k[[7, 150, 407], :, 0] = -3e38
    far, far_lse = _run(p, 1000)
    torch.cuda.synchronize()
    assert torch.equal(far_lse, lse) and torch.equal(far, weights)


@pytest.mark.parametrize("down", [60.0, 91.0, 100.0, 250.0])
def test_weights_beyond_the_largest_number_are_infinite(down, cuda_device):
    """An lse that is not the attention's own: terms up to exp(down) and past 2^128, where a
    sum is +inf, as the formula's is in 32 bits; never a finite number that is not it."""
    p = Prompt(cuda_device, (400, 70), 8, 2, 128, "bf16", 78)
    lse, scale = _lse(p, 1.0)            # few terms a key are near the largest
    low = lse - down
    weights = torch.full((2, 2, 400), 7.0, device=cuda_device)
    pa_prompt_weights(weights, p.q, p.k, low, p.starts, scale, 400)
    torch.cuda.synchronize()
    pa_check_error()
    top, seen = float(torch.finfo(torch.float32).max), 0
    for s, (b, n) in enumerate(((0, 400), (400, 70))):
        later = torch.ones((n, n), dtype=torch.bool, device=cuda_device).triu(1)
        for kv in range(2):
            k = p.k[b:b + n, kv].double()
            want, lim = torch.zeros(n, device=cuda_device).double(), 0.0
            for h in range(4 * kv, 4 * kv + 4):
                q = p.q[b:b + n, h].double()
                z = (q @ k.T * scale).masked_fill(later, -torch.inf)
                size = (q.abs() @ k.abs().T * scale).masked_fill(later, 0)
                x = (z - low[b:b + n, h, None].double()).exp()
                rel = (p.D * 2.0 ** -23 * size + 4 * 2.0 ** -24 * (z.abs().masked_fill(later, 0) +
                       low[b:b + n, h, None].abs()) + 2.0 ** -21 + (40 + 4 * n // 100) * 2.0 ** -24)
                want, lim = want + x.sum(0), lim + (x * rel).sum(0)
            got = weights[s, kv, :n].double()
            assert (got[want > top + lim] == torch.inf).all()
            fits = want < top - lim
            assert ((got - want).abs()[fits] <= lim[fits]).all()
            seen += int((want > top + lim).sum())
    assert (seen > 0) == (down > 80)


@pytest.mark.parametrize("at,value,left_out", [(3, 171, 2), (0, -1, 0), (0, 41, 0)])
def test_bad_bounds_alone_are_reported_and_left_out(at, value, left_out, cuda_device):
    """Every sequence fits the columns: only the bounds are wrong."""
    p = Prompt(cuda_device, (40, 70, 60), 4, 2, 64, "f16", 81)
    lse, scale = _lse(p)
    weights = torch.full((3, 2, 80), 7.0, device=cuda_device)
    right = int(p.starts[at])
    p.starts[at] = value
    pa_prompt_weights(weights, p.q, p.k, lse, p.starts, scale, 8)
    with pytest.raises(PagedAttentionError, match=f"query, index {left_out}"):
        pa_check_error()
    assert (weights[left_out] == 7).all()
    p.starts[at] = right
    _check(p, weights, lse, 8, seqs=[s for s in range(3) if s != left_out])
