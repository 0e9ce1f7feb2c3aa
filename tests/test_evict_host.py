"""Refusals of the eviction calls, on the host (CPU only)."""
import pytest
import torch

from paged_kv_cache_444_b200 import (EvictionState, _lib, pa_evict_commit, pa_evict_compact,
                                     pa_evict_select)

OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP, CUDA, BOUNDS = range(8)
FAKE = 0x10000

host_only = pytest.mark.skipif(torch.cuda.is_available(),
                               reason="stand-in pointers: host-only validation test")


def _call(name, order, base, **kw):
    args = dict(base)
    assert set(kw) <= set(args)
    args.update(kw)
    return getattr(_lib.load(), name)(*(args[k] for k in order), None)


SELECT_ORDER = ("source new_lens weights positions ctx recorded seq S Hk W B sink recent").split()
SELECT_BASE = dict({k: FAKE for k in SELECT_ORDER[:7]}, S=4, Hk=2, W=100, B=32, sink=4, recent=8)
COMPACT_ORDER = ("kc vc weights positions source new_lens bt ctx recorded seq S Hk D NB bs MB W B "
                 "eb").split()
COMPACT_BASE = dict({k: FAKE for k in COMPACT_ORDER[:10]}, S=4, Hk=2, D=128, NB=64, bs=16, MB=8,
                    W=100, B=32, eb=2)


@host_only
@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(S=-1)), (SHAPE, dict(Hk=0)), (SHAPE, dict(W=0)), (SHAPE, dict(B=0)),
    (SHAPE, dict(sink=-1)), (SHAPE, dict(recent=-1)), (SHAPE, dict(sink=25)),
    (SHAPE, dict(sink=33, recent=0)), (SHAPE, dict(S=1 << 28, Hk=2)),
    (UNSUP, dict(W=(1 << 19) + 1)), (NULL, dict(weights=None)), (NULL, dict(seq=None)),
    (ALIGN, dict(source=FAKE + 2)), (OK, dict(S=0, source=None)), (CUDA, dict()),
    (CUDA, dict(sink=24)),
])
def test_select_refusals(want, kw):
    assert _call("pa_evict_select", SELECT_ORDER, SELECT_BASE, **kw) == want


@host_only
@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(S=-1)), (SHAPE, dict(D=0)), (SHAPE, dict(eb=4)), (SHAPE, dict(bs=0)),
    (SHAPE, dict(NB=1 << 28)), (SHAPE, dict(MB=1 << 28)), (SHAPE, dict(B=1 << 31)),
    (UNSUP, dict(W=(1 << 19) + 1)), (NULL, dict(kc=None)), (NULL, dict(bt=None)),
    (NULL, dict(new_lens=None)), (ALIGN, dict(D=4)), (ALIGN, dict(D=8, eb=1)),
    (ALIGN, dict(vc=FAKE + 8)), (ALIGN, dict(bt=FAKE + 2)), (ALIGN, dict(positions=FAKE + 1)),
    (OK, dict(S=0)), (CUDA, dict()),
])
def test_compact_refusals(want, kw):
    assert _call("pa_evict_compact", COMPACT_ORDER, COMPACT_BASE, **kw) == want


def test_binding_refuses_wrong_tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = dict(source=i32(2, 3, 8), new_lens=i32(2), weights=torch.zeros(2, 3, 20),
                positions=i32(2, 3, 20), context_lens=i32(2), recorded_lens=i32(2),
                seq_lens=i32(2))
    lens = good["context_lens"]
    for bad in (dict(weights=torch.zeros(2, 3, 20).half()), dict(weights=torch.zeros(3, 20)),
                dict(weights=torch.zeros(2, 20, 3).transpose(1, 2)), dict(positions=i32(2, 3, 19)),
                dict(source=i32(2, 2, 8)), dict(source=torch.zeros(2, 3, 8, dtype=torch.int64)),
                dict(new_lens=i32(3)), dict(seq_lens=torch.zeros(2, dtype=torch.int64)),
                dict(new_lens=lens),                 # in place: other heads still read it
                {}):                                 # host tensors
        with pytest.raises(ValueError):
            pa_evict_select(**{**good, **bad}, sink=1, recent=2)
    kc = torch.zeros(4, 16, 3, 64, dtype=torch.float16)
    more = dict(key_cache=kc, value_cache=kc.clone(), block_tables=i32(2, 2))
    for bad in (dict(value_cache=torch.zeros(4, 16, 3, 32, dtype=torch.float16)),
                dict(key_cache=torch.zeros(4, 16, 2, 64, dtype=torch.float16)),
                dict(value_cache=kc.bfloat16()), dict(block_tables=i32(3, 2)),
                dict(block_tables=i32(2, 4)[:, ::2]), {}):
        with pytest.raises(ValueError):
            pa_evict_compact(**{**good, **more, **bad})


WEIGHTS_ORDER = ("out weights ws ws_bytes query kc vc bt ctx scale S H Hk D NB bs MB W new "
                 "dt").split()
WEIGHTS_BASE = dict({k: FAKE for k in ("out", "weights", "ws", "query", "kc", "vc", "bt", "ctx")},
                    ws_bytes=1 << 30, scale=0.1, S=4, H=8, Hk=2, D=128, NB=64, bs=16, MB=8, W=128,
                    new=1, dt=0)


@host_only
@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dt=7)), (SHAPE, dict(S=-1)), (SHAPE, dict(H=7)), (SHAPE, dict(W=0)),
    (SHAPE, dict(new=-1)), (SHAPE, dict(ws_bytes=100)), (SHAPE, dict(scale=float("inf"))),
    (NULL, dict(weights=None)), (NULL, dict(ws=None)), (NULL, dict(out=None)),
    (ALIGN, dict(ws=FAKE + 128)), (ALIGN, dict(weights=FAKE + 2)), (ALIGN, dict(out=FAKE + 8)),
    (UNSUP, dict(D=96)), (UNSUP, dict(bs=8)), (UNSUP, dict(H=64, Hk=2)),
    (OK, dict(S=0, ws=None)), (CUDA, dict()),
])
def test_decode_weights_refusals(want, kw):
    assert _call("pa_decode_weights", WEIGHTS_ORDER, WEIGHTS_BASE, **kw) == want


def test_decode_weights_workspace_bytes():
    f = _lib.load().pa_decode_weights_workspace_bytes
    # 4 x 8 rows of one 512-token partition (D + 2 floats), 128 logits each
    assert f(4, 8, 128, 8, 16) == 32 * 128 * 4 + 256 + 256 + 32 * 128 * 4
    assert f(0, 8, 128, 8, 16) == 0
    for bad in ((-1, 8, 128, 8, 16), (1, 0, 128, 8, 16), (1, 8, 0, 8, 16), (1, 8, 128, 0, 16)):
        assert f(*bad) == -1


PROMPT_ORDER = "out lse q k v qs ks vs starts scale S T H Hk D dt".split()
PROMPT_BASE = dict({k: FAKE for k in ("out", "lse", "q", "k", "v", "starts")}, qs=1024, ks=256,
                   vs=256, scale=0.1, S=3, T=100, H=8, Hk=2, D=128, dt=1)


@host_only
@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dt=2)), (SHAPE, dict(S=-1)), (SHAPE, dict(T=-1)), (SHAPE, dict(H=7)),
    (SHAPE, dict(qs=1016)), (SHAPE, dict(ks=128)), (SHAPE, dict(T=1 << 29)),
    (SHAPE, dict(scale=float("nan"))), (UNSUP, dict(D=96, qs=768)), (UNSUP, dict(H=64, Hk=2)),
    (NULL, dict(out=None)), (NULL, dict(v=None)), (NULL, dict(starts=None)),
    (ALIGN, dict(ks=260)), (ALIGN, dict(v=FAKE + 8)), (ALIGN, dict(lse=FAKE + 2)),
    (ALIGN, dict(D=68)), (OK, dict(S=0, q=None)), (OK, dict(T=0, q=None)),
    (CUDA, dict()), (CUDA, dict(lse=None)),
])
def test_prompt_refusals(want, kw):
    assert _call("pa_prompt_attention", PROMPT_ORDER, PROMPT_BASE, **kw) == want


PW_ORDER = "weights q k lse qs ks starts scale S T H Hk D W window dt".split()
PW_BASE = dict({k: FAKE for k in ("weights", "q", "k", "lse", "starts")}, qs=1024, ks=256,
               scale=0.1, S=3, T=100, H=8, Hk=2, D=128, W=50, window=8, dt=1)


@host_only
@pytest.mark.parametrize("want,kw", [
    (DTYPE, dict(dt=2)), (SHAPE, dict(S=-1)), (SHAPE, dict(window=0)), (SHAPE, dict(W=0)),
    (SHAPE, dict(ks=128)), (UNSUP, dict(H=64, Hk=2)), (NULL, dict(lse=None)),
    (NULL, dict(weights=None)), (NULL, dict(q=None)), (ALIGN, dict(qs=1028)),
    (ALIGN, dict(lse=FAKE + 1)), (ALIGN, dict(k=FAKE + 4)), (OK, dict(S=0)), (OK, dict(T=0)),
    (CUDA, dict()), (CUDA, dict(window=1 << 40)),
])
def test_prompt_weights_refusals(want, kw):
    assert _call("pa_prompt_weights", PW_ORDER, PW_BASE, **kw) == want


def test_a_workspace_serves_smaller_calls():
    """Fewer sequences or narrower tables never need more."""
    from paged_kv_cache_444_b200._lib import load
    size = load().pa_decode_weights_workspace_bytes
    for H, D in ((32, 128), (5, 64), (64, 64)):
        last = 0
        for S in range(0, 300):
            n = size(S, H, D, 40, 16)
            assert n >= last
            last = n
        last = 0
        for MB in range(1, 700):
            n = size(7, H, D, MB, 16)
            assert n >= last
            last = n


def test_eviction_state_refuses_a_budget_that_cannot_hold():
    EvictionState(1, 1, 32, 8, "cpu", sink=3, recent=5)
    for bad in (dict(sink=4, recent=5), dict(sink=9), dict(sink=-1), dict(recent=-1)):
        with pytest.raises(ValueError):
            EvictionState(1, 1, 32, 8, "cpu", **bad)


def test_eviction_state_refuses_lengths_in_one_tensor():
    """The new lengths would overwrite the tokens a sequence has had."""
    state = EvictionState(2, 1, 32, 8, "cpu")
    kc = torch.zeros(4, 16, 1, 64, dtype=torch.float16)
    lens = torch.full((2,), 20, dtype=torch.int32)
    with pytest.raises(ValueError, match="seq_lens must not share"):
        state.evict(kc, kc.clone(), torch.zeros(2, 2, dtype=torch.int32), lens, lens)


@pytest.mark.parametrize("apart", [-3, -1, 0, 1, 3])
def test_lengths_may_not_overlap_in_part(apart):
    """Views into one buffer a few entries apart: written in place, the same as one tensor."""
    buf = torch.zeros(12, dtype=torch.int32)
    one, other = buf[4:8], buf[4 + apart:8 + apart]
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = dict(source=i32(4, 1, 8), new_lens=one, weights=torch.zeros(4, 1, 20),
                positions=i32(4, 1, 20), context_lens=i32(4), recorded_lens=i32(4),
                seq_lens=i32(4))
    for name in ("context_lens", "recorded_lens", "seq_lens"):
        with pytest.raises(ValueError, match="new_lens must not share"):
            pa_evict_select(**{**good, name: other}, sink=1, recent=2)
    state = EvictionState(4, 1, 32, 8, "cpu")
    kc = torch.zeros(4, 16, 1, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="seq_lens must not share"):
        state.evict(kc, kc.clone(), i32(4, 2), one, other)


def test_lengths_side_by_side_are_apart():
    """Views that touch without a common entry go on to the next check (host tensors)."""
    buf = torch.zeros(16, dtype=torch.int32)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError, match="one CUDA device"):
        pa_evict_select(source=i32(4, 1, 8), new_lens=buf[4:8], weights=torch.zeros(4, 1, 20),
                        positions=i32(4, 1, 20), context_lens=buf[:4], recorded_lens=buf[8:12],
                        seq_lens=buf[12:], sink=1, recent=2)
    state = EvictionState(4, 1, 32, 8, "cpu")
    kc = torch.zeros(4, 16, 1, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="one CUDA device"):
        state.evict(kc, kc.clone(), i32(4, 2), buf[:4], buf[4:8])


COMMIT_ORDER = ("ctx", "recorded", "new_lens", "S")
COMMIT_BASE = dict(ctx=FAKE, recorded=FAKE + 64, new_lens=FAKE + 128, S=4)


@host_only
@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(S=-1)), (SHAPE, dict(S=1 << 31)), (NULL, dict(ctx=None)),
    (NULL, dict(recorded=None)), (NULL, dict(new_lens=None)), (ALIGN, dict(ctx=FAKE + 2)),
    (OK, dict(S=0, ctx=None)), (CUDA, dict()),
])
def test_commit_refusals(want, kw):
    assert _call("pa_evict_commit", COMMIT_ORDER, COMMIT_BASE, **kw) == want


def test_commit_binding_refuses_wrong_tensors():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    good = dict(context_lens=i32(3), recorded_lens=i32(3), new_lens=i32(3))
    buf = i32(8)
    for bad in (dict(context_lens=i32(4)), dict(recorded_lens=i32(3).long()),
                dict(new_lens=i32(6)[::2]), dict(new_lens=i32(3, 1)),
                dict(context_lens=buf[:3], new_lens=buf[2:5]),
                dict(context_lens=buf[:3], recorded_lens=buf[:3]), {}):      # (host tensors)
        with pytest.raises(ValueError):
            pa_evict_commit(**{**good, **bad})
