"""Cases and plain forms of the heavy-hitter cache operators: whole-prompt
attention over packed sequences, the attention weight each cached token has
received (from a prompt, and from decode steps), the selection of the tokens a
bounded cache keeps, and the move that packs them to the front of the paged
cache.

`run` computes an operator either in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or, with `own` set, through
the calls of the paged_kv_cache_444_b200 package.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
PAGE = 16
ROWS = 2048   # query rows the plain prompt attention holds logits for at a time


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def listed():
    return [
        # a few very short prompts, where the launch is the cost
        dict(name="prompt_tiny", op="prompt", dtype="f16", heads=4, kv_heads=4, dim=64,
             lens="1,9,16,37", fused=False),
        # a server's prompt batch of mixed lengths, rows of one fused QKV projection
        dict(name="prompt_packed_gqa", op="prompt", dtype="bf16", heads=32, kv_heads=8, dim=128,
             lens="513,4001,77,1210,2048,900,3500,640", fused=True),
        # one long document
        dict(name="prompt_long_gqa", op="prompt", dtype="bf16", heads=32, kv_heads=8, dim=128,
             lens="16384", fused=False),
        # what the last 32 tokens of each packed prompt look at (a short observation window)
        dict(name="prompt_weights_window", op="prompt_weights", dtype="bf16", heads=32,
             kv_heads=8, dim=128, lens="513,4001,77,1210,2048,900,3500,640", window=32,
             fused=True),
        # what every token of a prompt looks at, MHA
        dict(name="prompt_weights_whole", op="prompt_weights", dtype="f16", heads=32,
             kv_heads=32, dim=128, lens="4096,1333", window=4096, fused=False),
        # one decode step of four short sequences
        dict(name="decode_weights_tiny", op="decode_weights", dtype="f16", heads=4, kv_heads=4,
             dim=64, lens="1,9,16,37"),
        # a decode step over a large batch
        dict(name="decode_weights_gqa", op="decode_weights", dtype="bf16", heads=32, kv_heads=8,
             dim=128, lens="uniform:128:512:4096"),
        # a decode step over long contexts, before their first eviction
        dict(name="decode_weights_long", op="decode_weights", dtype="bf16", heads=32, kv_heads=8,
             dim=128, lens="uniform:8:32768:131072"),
        # the eviction every 17 decode steps of a batch that is held to 1000 tokens
        dict(name="select_steady", op="select", heads=32, kv_heads=8, dim=128, dtype="bf16",
             lens="fixed:128:1017", budget=1000, sink=4, recent=100, evicted=True),
        # the first eviction after long prompts
        dict(name="select_long", op="select", heads=32, kv_heads=8, dim=128, dtype="bf16",
             lens="uniform:8:32768:131072", budget=4096, sink=4, recent=512, evicted=False),
        # moving what the two evictions above keep
        dict(name="compact_steady", op="compact", heads=32, kv_heads=8, dim=128, dtype="bf16",
             lens="fixed:128:1017", budget=1000, sink=4, recent=100, evicted=True),
        dict(name="compact_long", op="compact", heads=32, kv_heads=8, dim=128, dtype="bf16",
             lens="uniform:8:32768:131072", budget=4096, sink=4, recent=512, evicted=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["prompt", "prompt_weights", "decode_weights", "select", "compact"])
    heads, kv_heads = rng.choice([(32, 8), (32, 32), (16, 2), (12, 4), (4, 4), (8, 1), (16, 1)])
    case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), heads=heads, kv_heads=kv_heads,
                dim=rng.choice([64, 128, 128]))
    if op in ("prompt", "prompt_weights"):
        total, lens = _log(rng, 1, 16384), []
        while total > 0 and len(lens) < 12:
            n = min(total, _log(rng, 1, 16384))
            lens.append(n)
            total -= n
        case.update(lens=",".join(map(str, lens)), fused=rng.random() < 0.5)
        if op == "prompt_weights":
            case["window"] = min(_log(rng, 1, 4096), max(lens))
    elif op == "decode_weights":
        seqs = _log(rng, 1, 200)
        hi = _log(rng, 1, min(131072, 600000 * 8 // (seqs * kv_heads)))
        case["lens"] = "uniform:%d:%d:%d" % (seqs, max(1, hi // rng.choice([1, 3, 8])), hi)
    else:
        budget = _log(rng, 16, 8192)
        evicted = rng.random() < 0.5
        seqs = _log(rng, 1, min(128, 100000 // budget + 1))
        if evicted:
            case["lens"] = "fixed:%d:%d" % (seqs, budget + _log(rng, 1, 64))
        else:
            hi = _log(rng, budget // 2 + 1, max(budget, min(131072, 400000 // seqs)))
            case["lens"] = "uniform:%d:%d:%d" % (seqs, max(1, hi // 4), hi)
        case.update(budget=budget, sink=rng.randint(0, 4), recent=rng.randint(1, budget // 2),
                    evicted=evicted)
    return case


def _lens(case):
    """Sequence lengths of a case: listed one by one, or a number of them all
    alike ("fixed") or spread evenly over a range ("uniform", shuffled)."""
    text = case["lens"]
    if ":" not in text:
        return [int(x) for x in text.split(",")]
    kind, *nums = text.split(":")
    nums = [int(x) for x in nums]
    if kind == "fixed":
        return [nums[1]] * nums[0]
    n, lo, hi = nums
    lens = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]
    random.Random(n * 7919 + hi).shuffle(lens)
    return lens


def _moves(case, n):
    """Expected rows one (sequence, KV head) moves, for weights without order."""
    budget, sink = case["budget"], case["sink"]
    if n <= budget:
        return 0
    if case["evicted"]:
        return min(n - budget, case["recent"])
    free = n - sink - case["recent"]
    heavy = max(0, budget - sink - case["recent"])
    return (budget - sink) * (1 - heavy / free)


def work(case):
    lens, H, Hk, D = _lens(case), case["heads"], case["kv_heads"], case["dim"]
    op, total, S = case["op"], sum(lens), len(lens)
    if op == "prompt":
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": total * (2 * H + 2 * Hk) * D * 2 + total * H * 4 + 4 * (S + 1),
                "flops": 4 * D * H * pairs}
    if op == "prompt_weights":
        rows = [min(n, case["window"]) for n in lens]
        pairs = sum(w * n - w * (w - 1) // 2 for w, n in zip(rows, lens))
        return {"bytes": sum(rows) * H * (D * 2 + 4) + total * Hk * (D * 2 + 4) + 4 * (S + 1),
                "flops": 2 * D * H * pairs}
    if op == "decode_weights":
        return {"bytes": total * Hk * (4 * D + 8) + 2 * S * H * D * 2 +
                4 * sum((n + PAGE - 1) // PAGE for n in lens) + 4 * S,
                "flops": 4 * D * H * total}
    kept = sum(min(n, case["budget"]) for n in lens)
    if op == "select":
        seen = kept if case["evicted"] else 0
        return {"bytes": Hk * 4 * (total + seen + S * case["budget"]) + 16 * S, "flops": 0}
    moved = sum(_moves(case, n) for n in lens)
    return {"bytes": Hk * (4 * S * case["budget"] + moved * (2 * 2 * D * 2 + 2 * 8) +
                           4 * (0 if case["evicted"] else kept)) + 16 * S,
            "flops": 0}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _prompt_state(case, gen):
    lens, dt = _lens(case), DTYPES[case["dtype"]]
    H, Hk, D, T = case["heads"], case["kv_heads"], case["dim"], sum(lens)
    if case["fused"]:     # one projection's rows: q, then k, then v of a token side by side
        qkv = _normal((T, H + 2 * Hk, D), dt, gen)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    else:
        q, k, v = (_normal((T, h, D), dt, gen) for h in (H, Hk, Hk))
    starts = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    return dict(case=case, q=q, k=k, v=v, starts=starts, lens=lens, scale=1 / math.sqrt(D))


def _tables(lens, gen):
    """Block tables of a paged cache: ids drawn without repeats, -1 past each sequence's end."""
    need = torch.tensor([(n + PAGE - 1) // PAGE for n in lens], device="cuda")
    width, blocks = int(need.max()), int(need.sum())
    perm = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    live = col[None] < need[:, None]
    at = (need.cumsum(0) - need)[:, None] + col[None]
    return torch.where(live, perm[at.clamp(max=blocks - 1)], -1).contiguous(), blocks


def _evict_state(case, gen):
    lens, Hk = _lens(case), case["kv_heads"]
    S, W, B = len(lens), max(lens), case["budget"]
    n = torch.tensor(lens, device="cuda")
    weights = torch.exp(1.5 * torch.randn((S, Hk, W), generator=gen, device="cuda"))
    st = dict(case=case, weights=weights, context_lens=n.to(torch.int32))
    slot = torch.arange(W, device="cuda")
    if case["evicted"]:
        # an earlier eviction left `budget` tokens of a sequence 50 times as long, sinks in
        # front and the others in no order; the tokens since then follow in their order
        length = n * 50
        since = (n - B)[:, None, None]
        old = torch.rand((S, Hk, W), generator=gen, device="cuda").argsort(-1)
        spread = case["sink"] + (old * ((length[:, None, None] - since - case["sink"]) // W))
        pos = torch.where(slot < case["sink"], slot, spread)
        st["recorded_lens"] = torch.full((S,), B, dtype=torch.int32, device="cuda")
    else:
        length, pos = n, torch.zeros((S, Hk, W), dtype=torch.int64, device="cuda")
        st["recorded_lens"] = torch.zeros(S, dtype=torch.int32, device="cuda")
    st["positions"] = pos.to(torch.int32).contiguous()
    st["seq_lens"] = length.to(torch.int32)
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dim = case["op"], case["dim"]
    dt = DTYPES[case["dtype"]]
    if op in ("prompt", "prompt_weights"):
        st = _prompt_state(case, gen)
        T, H = st["q"].shape[:2]
        if op == "prompt":
            st["out"] = torch.empty((T, H, dim), dtype=dt, device="cuda")
            st["lse"] = torch.empty((T, H), device="cuda")
        else:   # the attention's own log-sum-exp, which the weights are taken against
            st["lse"] = _plain_prompt(st)["lse"]
            st["weights"] = torch.zeros((len(st["lens"]), st["k"].shape[1], max(st["lens"])),
                                        device="cuda")
        return st
    if op == "decode_weights":
        lens, H, Hk = _lens(case), case["heads"], case["kv_heads"]
        tables, blocks = _tables(lens, gen)
        cache = (blocks, PAGE, Hk, dim)
        return dict(case=case, scale=1 / math.sqrt(dim), tables=tables,
                    context_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                    key_cache=_normal(cache, dt, gen), value_cache=_normal(cache, dt, gen),
                    q=_normal((len(lens), H, dim), dt, gen),
                    out=torch.empty((len(lens), H, dim), dtype=dt, device="cuda"),
                    # what earlier steps gave each token
                    weights=torch.rand((len(lens), Hk, tables.shape[1] * PAGE), generator=gen,
                                       device="cuda"))
    st = _evict_state(case, gen)
    S, Hk = st["weights"].shape[:2]
    st["source"] = torch.empty((S, Hk, case["budget"]), dtype=torch.int32, device="cuda")
    st["new_lens"] = torch.empty(S, dtype=torch.int32, device="cuda")
    if op == "compact":
        got = _plain_select(st)
        st["source"], st["new_lens"] = got["source"], got["new_lens"]
        st["tables"], blocks = _tables(_lens(case), gen)
        cache = (blocks, PAGE, Hk, dim)
        st["key_cache"], st["value_cache"] = _normal(cache, dt, gen), _normal(cache, dt, gen)
    return st


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------
def _logits(st, s, lo, hi):
    """fp32 logits [Hk, G, hi - lo, n] of query rows lo..hi-1 of sequence s against its
    first hi keys, -inf where a key is later than the query."""
    b = sum(st["lens"][:s])
    H, D = st["q"].shape[1:]
    Hk = st["k"].shape[1]
    q = st["q"][b + lo:b + hi].float().view(hi - lo, Hk, H // Hk, D).permute(1, 2, 0, 3)
    k = st["k"][b:b + hi].float().permute(1, 2, 0)[:, None]
    z = torch.matmul(q, k) * st["scale"]
    at = torch.arange(hi, device="cuda")
    return z.masked_fill_(at[None] > at[lo:hi, None], -math.inf)


def _plain_prompt(st):
    T, H, D = st["q"].shape
    Hk = st["k"].shape[1]
    out = torch.empty((T, H, D), dtype=st["q"].dtype, device="cuda")
    lse = torch.empty((T, H), device="cuda")
    b = 0
    for s, n in enumerate(st["lens"]):
        for lo in range(0, n, ROWS):
            hi = min(n, lo + ROWS)
            z = _logits(st, s, lo, hi)
            m = z.amax(-1, keepdim=True)
            z.sub_(m).exp_()
            l = z.sum(-1, keepdim=True)
            v = st["v"][b:b + hi].float().permute(1, 0, 2)[:, None]
            o = torch.matmul(z, v) / l
            out[b + lo:b + hi] = o.permute(2, 0, 1, 3).reshape(hi - lo, H, D).to(out.dtype)
            lse[b + lo:b + hi] = (m + l.log()).squeeze(-1).permute(2, 0, 1).reshape(hi - lo, H)
        b += n
    return {"out": out, "lse": lse}


def _plain_prompt_weights(st):
    b, window = 0, st["case"]["window"]
    Hk = st["k"].shape[1]
    for s, n in enumerate(st["lens"]):
        got = torch.zeros((Hk, n), dtype=torch.float64, device="cuda")
        for lo in range(max(0, n - window), n, ROWS):
            hi = min(n, lo + ROWS)
            z = _logits(st, s, lo, hi)
            lse = st["lse"][b + lo:b + hi].view(hi - lo, Hk, -1).permute(1, 2, 0)[..., None]
            got[:, :hi] += z.sub_(lse).exp_().sum((1, 2), dtype=torch.float64)
        st["weights"][s, :, :n] = got.float()
        b += n
    return {"weights": st["weights"]}


def _rows(cache, tables, s, n):
    """The first n cached rows of sequence s, [n, Hk, D]."""
    return cache[tables[s, :(n + PAGE - 1) // PAGE].long()].flatten(0, 1)[:n]


def _plain_decode_weights(st):
    S, H, D = st["q"].shape
    Hk = st["key_cache"].shape[2]
    for s, n in enumerate(_lens(st["case"])):
        k = _rows(st["key_cache"], st["tables"], s, n).float().permute(1, 2, 0)
        v = _rows(st["value_cache"], st["tables"], s, n).float().permute(1, 0, 2)
        z = torch.matmul(st["q"][s].float().view(Hk, H // Hk, D), k) * st["scale"]
        z = (z - z.amax(-1, keepdim=True)).exp_()
        p = z / z.sum(-1, keepdim=True)
        st["out"][s] = torch.matmul(p, v).view(H, D).to(st["out"].dtype)
        got = p.sum(1)
        st["weights"][s, :, :n - 1] += got[:, :-1]     # the token of this step starts anew
        st["weights"][s, :, n - 1] = got[:, -1]
    return {"out": st["out"], "weights": st["weights"]}


def _position_of(st, n):
    """Position of every slot: recorded, or counted back from the sequence's length."""
    slot = torch.arange(st["weights"].shape[-1], device="cuda")
    late = (st["seq_lens"].long() - n)[:, None, None] + slot
    return torch.where(slot < st["recorded_lens"][:, None, None], st["positions"].long(), late)


def _plain_select(st):
    case, w = st["case"], st["weights"]
    W, B = w.shape[-1], case["budget"]
    n = st["context_lens"].long()
    new = n.clamp(max=B)
    slot = torch.arange(W, device="cuda")
    live = slot < n[:, None, None]
    pos, length = _position_of(st, n), st["seq_lens"].long()[:, None, None]
    held = (pos < case["sink"]) | (pos >= length - case["recent"])
    key = torch.where(held, math.inf, w).masked_fill(~live, -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., :B]
    kept = torch.zeros_like(live.expand_as(w)).scatter(-1, order, True) & live
    front = slot < new[:, None, None]
    tail = torch.where(kept & ~front, slot, W).sort(dim=-1).values[..., :B]
    hole = (front & ~kept)[..., :B]
    nth = (hole.long().cumsum(-1) - 1).clamp(min=0)
    source = torch.where(hole, tail.gather(-1, nth.clamp(max=tail.shape[-1] - 1)),
                         slot[:hole.shape[-1]])
    st["source"].fill_(-1)
    st["source"][..., :hole.shape[-1]] = source.masked_fill(~front[..., :B], -1).to(torch.int32)
    st["new_lens"].copy_(new)
    return {"source": st["source"], "new_lens": st["new_lens"]}


def _plain_compact(st):
    n, new = st["context_lens"].long(), st["new_lens"].long()
    source = st["source"].long()
    S, Hk, B = source.shape
    slot = torch.arange(B, device="cuda")
    pos = _position_of(st, n)
    live = slot < new[:, None, None]
    src = torch.where(live, source, 0)
    width = min(B, st["weights"].shape[-1])
    live, src = live[..., :width], src[..., :width]
    for name, values in (("weights", st["weights"]), ("positions", pos.to(torch.int32))):
        got = values.gather(-1, src)
        st[name][..., :width] = torch.where(live, got, st[name][..., :width])
    s, h, i = (live & (src != slot[:width])).nonzero(as_tuple=True)
    j, tables = src[s, h, i], st["tables"].long()
    for cache in (st["key_cache"], st["value_cache"]):
        cache[tables[s, i // PAGE], i % PAGE, h] = cache[tables[s, j // PAGE], j % PAGE, h]
    return {k: st[k] for k in ("key_cache", "value_cache", "weights", "positions")}


PLAIN = {"prompt": _plain_prompt, "prompt_weights": _plain_prompt_weights,
         "decode_weights": _plain_decode_weights, "select": _plain_select,
         "compact": _plain_compact}


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return PLAIN[state["case"]["op"]](state)


def _run_own(st):
    import paged_kv_cache_444_b200 as pa
    case = st["case"]
    op = case["op"]
    if op == "prompt":
        pa.pa_prompt_attention(st["out"], st["lse"], st["q"], st["k"], st["v"], st["starts"],
                               st["scale"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "prompt_weights":
        pa.pa_prompt_weights(st["weights"], st["q"], st["k"], st["lse"], st["starts"],
                             st["scale"], case["window"])
        return {"weights": st["weights"]}
    if op == "decode_weights":
        if "workspace" not in st:     # kept for every step of the program
            st["workspace"] = pa.WeightsWorkspace.for_call(st["q"], st["key_cache"], st["tables"])
        pa.pa_decode_weights(st["out"], st["weights"], st["workspace"], st["q"],
                             st["key_cache"], st["value_cache"], st["tables"],
                             st["context_lens"], st["scale"], 1)
        return {"out": st["out"], "weights": st["weights"]}
    if op == "select":
        pa.pa_evict_select(st["source"], st["new_lens"], st["weights"], st["positions"],
                           st["context_lens"], st["recorded_lens"], st["seq_lens"],
                           case["sink"], case["recent"])
        return {"source": st["source"], "new_lens": st["new_lens"]}
    pa.pa_evict_compact(st["key_cache"], st["value_cache"], st["weights"], st["positions"],
                        st["source"], st["new_lens"], st["tables"], st["context_lens"],
                        st["recorded_lens"], st["seq_lens"])
    return {k: st[k] for k in ("key_cache", "value_cache", "weights", "positions")}


# --------------------------------------------------------------------------
# From the definitions, in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "select":
        return None                     # whole numbers
    H, Hk = case["heads"], case["kv_heads"]
    f64 = torch.float64
    if op in ("prompt", "prompt_weights"):
        T = st["q"].shape[0]
        out = torch.zeros(st["q"].shape, dtype=f64, device="cuda")
        lse = torch.zeros((T, H), dtype=f64, device="cuda")
        weights = torch.zeros((len(st["lens"]), Hk, max(st["lens"])), dtype=f64, device="cuda")
        for s, n in enumerate(st["lens"]):
            b = sum(st["lens"][:s])
            first = n - min(n, case["window"]) if op == "prompt_weights" else 0
            later = torch.ones((n - first, n), dtype=torch.bool, device="cuda").triu(first + 1)
            for h in range(H):
                kv = h * Hk // H
                q, k = st["q"][b + first:b + n, h].to(f64), st["k"][b:b + n, kv].to(f64)
                z = (q @ k.T).mul_(st["scale"]).masked_fill_(later, -math.inf)
                if op == "prompt":
                    lse[b:b + n, h] = torch.logsumexp(z, -1)
                    out[b:b + n, h] = torch.softmax(z, -1) @ st["v"][b:b + n, kv].to(f64)
                else:      # against the log-sum-exp that the call is given
                    weights[s, kv, :n] += (z - st["lse"][b + first:b + n, h, None]).exp().sum(0)
        return {"out": out, "lse": lse} if op == "prompt" else {"weights": weights}
    if op == "decode_weights":
        out, weights = torch.zeros(st["q"].shape, dtype=f64, device="cuda"), st["weights"].to(f64)
        for s, n in enumerate(_lens(case)):
            at = torch.arange(n, device="cuda")
            block, row = st["tables"][s].long()[at // PAGE], at % PAGE
            weights[s, :, n - 1] = 0
            for h in range(H):
                kv = h * Hk // H
                k = st["key_cache"][block, row, kv].to(f64)
                p = torch.softmax(k @ st["q"][s, h].to(f64) * st["scale"], 0)
                out[s, h] = p @ st["value_cache"][block, row, kv].to(f64)
                weights[s, kv, :n] += p
        return {"out": out, "weights": weights}
    got = {k: st[k].clone() for k in ("key_cache", "value_cache", "weights")}
    src, new = st["source"].long(), st["new_lens"].tolist()
    for s in range(len(new)):
        for h in range(Hk):
            dst = (src[s, h, :new[s]] != torch.arange(new[s], device="cuda")).nonzero()[:, 0]
            frm = src[s, h, dst]
            got["weights"][s, h, dst] = st["weights"][s, h, frm]
            tab = st["tables"][s].long()
            for name in ("key_cache", "value_cache"):
                rows = st[name][tab[frm // PAGE], frm % PAGE, h]
                got[name][tab[dst // PAGE], dst % PAGE, h] = rows
    return {**{k: v.to(f64) for k, v in got.items()}, "positions": None}
