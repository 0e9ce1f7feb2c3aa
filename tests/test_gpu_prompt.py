"""pa_prompt_attention against causal attention in 64 bits, head by head."""
import numpy as np
import pytest
import torch

from paged_kv_cache_444_b200 import (PagedAttentionError, pa_check_error, pa_prefill,
                                     pa_prompt_attention, pa_reshape_and_cache)
from weights_reference import HALF, attend, out_bound

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


class Prompt:
    """Packed rows; `lead` and `trail` rows belong to no sequence (NaN)."""

    def __init__(self, dev, lens, H, Hk, D, dtype, seed, fused=False, lead=0, trail=0):
        g = torch.Generator(device=dev).manual_seed(seed)
        T = lead + sum(lens) + trail
        self.lens, self.H, self.Hk, self.D, self.T = lens, H, Hk, D, T
        if fused:
            x = torch.randn((T, H + 2 * Hk, D), generator=g, device=dev).to(DT[dtype])
            self.q, self.k, self.v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
        else:
            self.q, self.k, self.v = (torch.randn((T, h, D), generator=g, device=dev).to(DT[dtype])
                                      for h in (H, Hk, Hk))
        for x in (self.q, self.k, self.v):
            x[:lead] = float("nan")
            x[T - trail:] = float("nan")
        self.starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]) + lead,
                                   dtype=torch.int32, device=dev)
        self.out = torch.full((T, H, D), 7.0, dtype=DT[dtype], device=dev)
        self.lse = torch.full((T, H), 7.0, device=dev)

    def run(self, scale=None, stream=None):
        self.scale = self.D ** -0.5 if scale is None else scale
        pa_prompt_attention(self.out, self.lse, self.q, self.k, self.v, self.starts, self.scale,
                            stream)
        return self

    def check(self, seqs=None, heads=None, rows=None):
        """rows: only the first `rows` tokens of each sequence."""
        torch.cuda.synchronize()
        pa_check_error()
        starts, G = self.starts.tolist(), self.H // self.Hk
        for s in range(len(self.lens)) if seqs is None else seqs:
            b, n = starts[s], self.lens[s] if rows is None else min(rows, self.lens[s])
            if n == 0:
                continue
            for h in range(self.H) if heads is None else heads:
                v = self.v[b:b + n, h // G]
                _, o, lse, rel, pv = attend(self.q[b:b + n, h], self.k[b:b + n, h // G], v,
                                            self.scale, 0)
                lim = out_bound(o, pv, rel, n, float(v.double().abs().max()), self.out.dtype,
                                HALF[self.out.dtype])
                err = (self.out[b:b + n, h].double() - o).abs()
                assert (err <= lim).all(), (s, h, float((err / lim).max()))
                err = (self.lse[b:b + n, h].double() - lse).abs()
                # the sum is off by rel, log by 2^-22, the result rounded
                lim = rel + 2.0 ** -21 + 2.0 ** -23 * lse.abs() + n * 2.0 ** -23
                assert (err <= lim).all(), (s, h, float((err / lim).max()))
        lo, hi = starts[0], starts[-1]
        for x in (self.out, self.lse):     # rows of no sequence are left as they were
            assert (x[:lo] == 7).all() and (x[hi:] == 7).all()


CASES = {
    # name: (lengths, heads, KV heads, head_dim, dtype, options)
    "one_token": ((1,), 1, 1, 64, "f16", {}),
    "tiny": ((1, 9, 16, 37), 4, 4, 64, "f16", dict(trail=3)),
    "tile_edges_mha": ((127, 128, 129, 255, 256, 257), 2, 2, 128, "bf16", dict(lead=5)),
    "tile_edges_gqa4": ((31, 32, 33, 63, 64, 65, 127, 129), 8, 2, 128, "bf16", dict(fused=True)),
    "empty_between": ((0, 50, 0, 0, 70, 0), 8, 2, 64, "bf16", dict(lead=2, trail=9)),
    "group3": ((45, 200, 1), 12, 4, 128, "f16", dict(fused=True)),
    "group5_d64": ((130, 27), 5, 1, 64, "f16", dict(trail=1)),
    "group16": ((300, 50), 32, 2, 128, "bf16", {}),
    "group9": ((99, 140), 9, 1, 128, "bf16", {}),
    "mha_f16": ((200, 65, 129), 4, 4, 128, "f16", dict(fused=True)),
    "ragged_gqa4": ((513, 77, 1210, 640), 8, 2, 128, "bf16", dict(fused=True, trail=11)),
    "long_gqa8_d64": ((2500, 1100), 8, 1, 64, "f16", {}),
    # more pairs of tiles than SMs: two tiles an item (else one, in two halves)
    "pairs_mha_d64": ((2500, 1100, 700), 16, 16, 64, "f16", dict(trail=2)),
    "pairs_gqa4": ((1300, 900, 513), 32, 8, 128, "bf16", dict(fused=True, lead=3)),
    "pairs_group3": ((300, 41, 84, 85), 48, 16, 128, "f16", {}),
    "long_mha": ((1900, 1025), 2, 2, 128, "bf16", {}),
}


@pytest.mark.parametrize("name", CASES)
def test_matches_the_definition(name, cuda_device):
    lens, H, Hk, D, dtype, kw = CASES[name]
    Prompt(cuda_device, lens, H, Hk, D, dtype, 40 + len(name), **kw).run().check()


def _draw(seed, n, hi):
    return tuple(int(x) for x in np.random.default_rng(seed).integers(0, hi, n))


@pytest.mark.parametrize("lens,H,Hk,seqs", [
    (_draw(1, 256, 40), 4, 2, range(0, 256, 5)),       # the most that are ranked by length
    (_draw(2, 300, 40), 4, 2, range(0, 300, 7)),       # more: in their own order
    (_draw(3, 1200, 9), 4, 1, range(0, 1200, 31)),     # several sequences a thread
    ((129,) * 256, 16, 1, range(0, 256, 63)),          # few sequences, more units than are ranked
], ids=["256", "300", "1200", "units"])
def test_many_sequences(lens, H, Hk, seqs, cuda_device):
    p = Prompt(cuda_device, lens, H, Hk, 64, "bf16", 81).run()
    p.check(seqs)
    assert not (p.out == 7).all(-1).any() and not p.out.isnan().any()   # every row was written


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 0.0, -0.2])
def test_other_scales(scale, dtype, cuda_device):
    """1: peaked rows whose reference maximum moves between the key blocks."""
    Prompt(cuda_device, (900, 333), 8, 2, 128, dtype, 82).run(scale).check()
    Prompt(cuda_device, (900, 333), 32, 16, 128, dtype, 92).run(scale).check(heads=[0, 9, 31])


@pytest.mark.parametrize("H,Hk,dtype", [(2, 2, "bf16"), (8, 2, "f16"), (32, 32, "bf16")])
def test_climbing_logits(H, Hk, dtype, cuda_device):
    """Logits that climb by 10 log2 units every 64 keys, for half of the rows."""
    p = Prompt(cuda_device, (700, 100), H, Hk, 128, dtype, 83)
    u = torch.randn(128, device=cuda_device)
    u /= u.norm()
    at = torch.cat([torch.arange(n, device=cuda_device) for n in p.lens])
    p.k.copy_((p.k.float() * 0.25 + (7.0 * (at // 64))[:, None, None] * u).to(p.k.dtype))
    p.q[::2] = (p.q[::2].float() * 0.25 + u * 128 ** 0.5).to(p.q.dtype)
    p.run().check()


@pytest.mark.parametrize("dtype,H,Hk,D", [("bf16", 8, 2, 128), ("f16", 2, 2, 64),
                                            ("bf16", 64, 16, 128)])
def test_what_a_token_does_not_see_does_not_reach_it(dtype, H, Hk, D, cuda_device):
    """NaN and infinities in a later token's rows and in the next sequence's."""
    p = Prompt(cuda_device, (150, 90, 40, 260), H, Hk, D, dtype, 84)
    b = p.starts.tolist()
    p.k[b[1]:b[1] + 2] = float("nan")               # sequence 1: all of it
    p.v[b[1]:b[2]:7] = float("inf")
    p.v[b[0] + 100, 0, 3] = float("inf")            # sequence 0: tokens from 100 on
    p.v[b[0] + 120, 0, 3] = float("-inf")
    p.v[b[0] + 110, Hk - 1, D - 1] = float("nan")
    p.q[b[2] + 20] = float("nan")                   # sequence 2: that token alone
    p.k[b[3] + 200] = float("inf")                  # sequence 3: tokens from 200 on
    p.v[b[3] + 130, 0, 1] = float("nan")            # and dim 1 of head 0 from 130 on
    p.run()
    torch.cuda.synchronize()
    G = H // Hk
    o = p.out[b[0]:b[1]]
    assert (o[100:120, :G, 3] == float("inf")).all() and o[120:, :G, 3].isnan().all()
    assert o[110:, H - G:, D - 1].isnan().all() and o[:110, H - G:, D - 1].isfinite().all()
    fine = o.clone()
    fine[100:, :G, 3] = 0
    fine[110:, H - G:, D - 1] = 0
    assert fine.isfinite().all() and p.lse[b[0]:b[1]].isfinite().all()
    assert p.out[b[2] + 20].isnan().all() and p.lse[b[2] + 20].isnan().all()
    others = torch.cat([p.out[b[2]:b[2] + 20], p.out[b[2] + 21:b[3]]])
    assert others.isfinite().all()
    o = p.out[b[3]:b[4]]
    assert o[:130].isfinite().all() and o[130:200, :G, 1].isnan().all()
    fine = o[:200].clone()
    fine[130:, :G, 1] = 0
    assert fine.isfinite().all()
    p.check(seqs=[0], rows=100)
    p.check(seqs=[2], rows=20)
    p.check(seqs=[3], rows=130)


def test_lse_is_optional_and_rows_may_be_strided(cuda_device):
    p = Prompt(cuda_device, (140, 33), 8, 2, 128, "bf16", 85).run()
    wide = torch.full((p.T, 11, 128), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    k = wide[:, 3:5]
    k.copy_(p.k)
    out = torch.empty_like(p.out)
    pa_prompt_attention(out, None, p.q, k, p.v, p.starts, p.scale)
    assert torch.equal(out, p.out)
    p.check()


def test_agrees_with_the_prefill_over_the_cache(cuda_device):
    """The same prompts written to a paged cache and prefilled from it: two
    kernels within their roundings of one another (each within out_bound)."""
    lens = (300, 17, 129)
    p = Prompt(cuda_device, lens, 8, 2, 128, "f16", 86).run()
    blocks = sum(-(-n // 16) for n in lens)
    kc = torch.zeros((blocks, 16, 2, 128), dtype=torch.float16, device=cuda_device)
    vc = torch.zeros_like(kc)
    tables = torch.full((3, 19), -1, dtype=torch.int32)
    slots, at = [], 0
    for s, n in enumerate(lens):
        m = -(-n // 16)
        tables[s, :m] = torch.arange(at, at + m)
        slots += [at * 16 + i for i in range(n)]
        at += m
    pa_reshape_and_cache(p.k, p.v, kc, vc, torch.tensor(slots, device=cuda_device))
    out = torch.empty_like(p.out)
    pa_prefill(out, p.q, kc, vc, tables.to(cuda_device),
               torch.tensor(lens, dtype=torch.int32, device=cuda_device), p.starts, p.scale,
               max(lens))
    torch.cuda.synchronize()
    assert (out.float() - p.out.float()).abs().max() < 4e-3
    p.check()


@pytest.mark.parametrize("at,value,left_out", [(3, 151, 2), (0, -1, 0)])
def test_bad_bounds_are_reported_and_left_out(at, value, left_out, cuda_device):
    p = Prompt(cuda_device, (40, 50, 60), 4, 2, 64, "f16", 87)
    p.starts[at] = value
    p.run()
    with pytest.raises(PagedAttentionError, match=f"query, index {left_out}"):
        pa_check_error()
    first = [0, 40, 90, 150]
    assert (p.out[first[left_out]:first[left_out + 1]] == 7).all()
    p.starts.copy_(torch.tensor(first, dtype=torch.int32))
    p.check(seqs=[s for s in range(3) if s != left_out])


def test_graph_and_another_stream(cuda_device):
    p = Prompt(cuda_device, (140, 33, 500), 8, 2, 128, "bf16", 88)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.run(stream=side)
    side.synchronize()
    p.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    p.v.normal_()
    p.starts.copy_(torch.tensor([0, 100, 133, 673], dtype=torch.int32))   # other lengths, too
    p.lens = (100, 33, 540)
    graph.replay()
    p.check()


def test_binding_refuses(cuda_device):
    p = Prompt(cuda_device, (20,), 8, 2, 64, "f16", 89)
    a = dict(out=p.out, lse=p.lse, query=p.q, key=p.k, value=p.v, seq_starts=p.starts, scale=0.1)
    for bad in (dict(value=p.v[:, :1]), dict(key=p.k[:19], value=p.v[:19]),
                dict(key=p.k.bfloat16()), dict(out=p.out[:10]), dict(lse=p.lse.half()),
                dict(seq_starts=p.starts.long()), dict(key=p.k.cpu()),
                dict(query=p.q.transpose(0, 1)), dict(query=p.q[..., :32])):
        with pytest.raises(ValueError):
            pa_prompt_attention(**{**a, **bad})
    with pytest.raises(PagedAttentionError, match="PA_ERR_SHAPE"):
        pa_prompt_attention(**{**a, "scale": float("nan")})


def test_rows_whose_logits_are_all_minus_infinity(cuda_device):
    """A product beyond 32 bits: out 0 and lse -inf where a row sees nothing else, and no
    weight on such keys where it does."""
    p = Prompt(cuda_device, (300, 40), 4, 2, 64, "bf16", 88)
    p.q[:, :, 0] = 3e38
    p.k[:, :, 0] = 0
    p.k[:260] = 0
    p.k[:260, :, 0] = -3e38
    p.run()
    torch.cuda.synchronize()
    pa_check_error()
    assert (p.out[:260] == 0).all() and (p.lse[:260] == -torch.inf).all()
    p.check(seqs=[1])
    # the rows after them see keys 260.. alone
    tail = Prompt(cuda_device, (40,), 4, 2, 64, "bf16", 88)
    for name in "qkv":
        getattr(tail, name).copy_(getattr(p, name)[260:300])
    tail.scale = p.scale
    tail.out, tail.lse = p.out[260:300], p.lse[260:300]
    tail.check()


def test_offsets_beyond_32_bits(cuda_device):
    """140000 rows of 128 heads of 128 out of a fused projection: 2.3e9 elements of out."""
    p = Prompt(cuda_device, (1,), 128, 8, 128, "bf16", 89)
    lens, T = (1000,) * 140, 140000
    x = torch.empty((T, 144, 128), dtype=torch.bfloat16, device=cuda_device)
    x.normal_(generator=torch.Generator(device=cuda_device).manual_seed(90))
    p.lens, p.T, p.q, p.k, p.v = lens, T, x[:, :128], x[:, 128:136], x[:, 136:]
    p.starts = torch.arange(0, T + 1, 1000, dtype=torch.int32, device=cuda_device)
    p.out = torch.full((T, 128, 128), 7.0, dtype=torch.bfloat16, device=cuda_device)
    p.lse = torch.full((T, 128), 7.0, device=cuda_device)
    p.run().check(seqs=[0, 131, 139], heads=[0, 77, 127])


def test_a_single_kv_head_may_have_any_head_stride(cuda_device):
    p = Prompt(cuda_device, (70, 30), 4, 1, 64, "f16", 91)
    want = p.run().out.clone()
    wide = torch.zeros((100, 3, 64), dtype=torch.float16, device=cuda_device)
    wide[:, 1] = p.k[:, 0]
    p.k = wide.as_strided((100, 1, 64), (192, 8, 1), 64)      # one head: its stride says nothing
    p.run().check()
    assert torch.equal(p.out, want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,D", [(2, 64), (16, 64), (2, 128), (16, 128)])
def test_small_weights_beside_a_large_one(H, D, dtype, cuda_device):
    """One key takes nearly all of the weight and has no value; thousands of keys at 2^-25.7 to
    2^-26.4 of it make the output.  An fp16 P is below its normal numbers there: an error of
    2^-25 each, against a sum of at least 2^7 (P is held 2^7 up), is 2^-32 of a value."""
    n = 5000
    p = Prompt(cuda_device, (n,), H, H, D, dtype, 94)
    p.q.zero_()
    p.q[..., 0] = 8
    p.k.zero_()
    step = torch.arange(n, device=cuda_device)
    p.k[:, :, 0] = (-9.8125 - 0.25 * (step % 3))[:, None].to(p.k.dtype)
    p.k[0, :, 0] = 8
    p.v.copy_((500 + 500 * torch.rand(p.v.shape, device=cuda_device)).to(p.v.dtype))
    p.v[0] = 0
    p.run(0.125)
    torch.cuda.synchronize()
    pa_check_error()
    half, rows = HALF[p.out.dtype], 300
    for h in (0, H - 1):
        _, o, lse, rel, pv = attend(p.q[n - rows:, h], p.k[:, h], p.v[:, h], 0.125, n - rows)
        lim = (half * o.abs() + (half + 2 * rel[:, None] + n * 2.0 ** -23) * pv +
               (n * 2.0 ** -32 * 1000 + 2.0 ** -25) * (dtype == "f16")) * (1 + half)
        err = (p.out[n - rows:, h].double() - o).abs()
        assert (err <= lim).all(), (h, float((err / lim).max()))
        err = (p.lse[n - rows:, h].double() - lse).abs()
        assert (err <= rel + 2.0 ** -21 + 2.0 ** -23 * lse.abs() + n * 2.0 ** -23).all()
