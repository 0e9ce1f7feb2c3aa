"""The steps on a stream that is not the current one: what they allocate must not
be memory that the other stream may still use, or be given next."""
import pytest
import torch

import paged_kv_cache_444_b200 as pa
from paged_kv_cache_444_b200 import workloads

pytestmark = pytest.mark.gpu
BUSY = 50_000_000            # cycles of a spinning kernel, some 25 ms


def _busy(stream):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(BUSY)


def _prompt(dev):
    g = torch.Generator(device=dev).manual_seed(5)
    q, k, v = (torch.randn((900, h, 64), generator=g, device=dev).half() for h in (8, 2, 2))
    starts = torch.tensor([0, 500, 900], dtype=torch.int32, device=dev)
    return dict(query=q, key=k, value=v, key_cache=None, value_cache=None, slot_mapping=None,
                seq_starts=starts, scale=0.125)


class _Wrapped:
    """Another library's stream: all that is known of it is its handle."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


def _handles(stream):
    return {"torch": stream, "handle": stream.cuda_stream, "wrapped": _Wrapped(stream)}


@pytest.mark.parametrize("kind", ["torch", "handle", "wrapped"])
def test_prompt_step_owns_what_it_allocates(kind, cuda_device, monkeypatch):
    """The log-sum-exp lives until the given stream has read it, and the output is
    nothing that the current stream still uses."""
    a = _prompt(cuda_device)
    weights = torch.zeros((2, 2, 500), device=cuda_device)
    want = torch.zeros_like(weights)
    want_out = pa.prompt_step(**a, weights=want, window=500)
    lse_at, real = [], pa.pa_prompt_weights

    def spy(weights, query, key, lse, *rest):
        lse_at.append(lse.data_ptr())
        return real(weights, query, key, lse, *rest)

    monkeypatch.setattr(pa, "pa_prompt_weights", spy)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    side.wait_stream(here)
    # freed here while this stream has yet to use it
    torch.cuda._sleep(BUSY)
    used = torch.empty_like(want_out)
    used.fill_(3)
    used_at = used.data_ptr()
    del used
    _busy(side)
    out = pa.prompt_step(**a, weights=weights, window=500, stream=_handles(side)[kind])
    assert out.data_ptr() != used_at
    later = [torch.full((900, 8), 1e30, device=cuda_device) for _ in range(4)]
    assert lse_at[0] not in [t.data_ptr() for t in later]
    torch.cuda.synchronize()
    pa.pa_check_error()
    assert torch.equal(weights, want) and torch.equal(out, want_out)
    # used on the current stream, then freed: not handed to `side` before that is done
    torch.cuda._sleep(BUSY)
    copy, at = out.clone(), out.data_ptr()
    del out
    again = pa.prompt_step(**a, stream=_handles(side)[kind])
    assert again.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(copy, want_out) and torch.equal(again, want_out)


def test_prompt_step_on_the_default_stream_by_handle(cuda_device):
    a = _prompt(cuda_device)
    want = pa.prompt_step(**a)
    assert torch.equal(pa.prompt_step(**a, stream=0), want)
    torch.cuda.synchronize()
    pa.pa_check_error()


@pytest.mark.parametrize("kind", ["torch", "handle", "wrapped"])
def test_decode_step_owns_what_it_allocates(kind, cuda_device, monkeypatch):
    """The same for decode_step: its output, and the workspace of the split form."""
    cfg = workloads.CONFIGS["tiny"]
    b = workloads.make_batch(cfg, cuda_device)
    a = (b.query, b.key, b.value, b.key_cache, b.value_cache, b.slot_mapping, b.block_tables,
         b.context_lens, cfg.scale)
    want = pa.decode_step(*a, partition_size=16)
    tmp, real = [], pa.pa_decode_split

    def spy(tmp_out, *rest):
        tmp.append(tmp_out)
        return real(tmp_out, *rest)

    monkeypatch.setattr(pa, "pa_decode_split", spy)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    used = torch.empty_like(want)
    used.fill_(3)
    used_at = used.data_ptr()
    del used
    _busy(side)
    out = pa.decode_step(*a, partition_size=16, stream=_handles(side)[kind])
    assert out.data_ptr() != used_at
    shape, dtype, tmp_at = tmp[0].shape, tmp[0].dtype, tmp.pop().data_ptr()
    later = [torch.full(shape, 1e30, dtype=dtype, device=cuda_device) for _ in range(4)]
    assert tmp_at not in [t.data_ptr() for t in later]
    torch.cuda.synchronize()
    pa.pa_check_error()
    assert torch.equal(out, want)
