"""Attention over a paged cache of keys and values, as cases to measure.

Three operators take a batch of requests of any lengths from its lengths to the rows that the output
projection reads:

  tables     block tables, slots and positions of a step's tokens from the requests' lengths (moe_lora_page_tables)
  write      new keys and values into their slots of the cache                                (moe_lora_cache_write)
  attention  causal attention of the new tokens to their requests' pages                     (moe_lora_attention)

Where `own` is false `run` computes them from elementary torch operations (attention in 32 bits on
the batch padded to its longest request); where it is true it calls the framework.  `exact` computes
them request by request, in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

_handle = None


def _pkg():
    import routed_moe_expert_gb300 as pkg
    return pkg


def _the_handle():
    """The library handle that a program creates once and keeps."""
    global _handle
    if _handle is None:
        _handle = _pkg().Handle(torch.cuda.current_device())
    return _handle


# ------------------------------------------------------------------------------------ the cases
# `lengths` seeds the requests' lengths: `chunks` requests bring `chunk` new tokens each (prompts, or
# pieces of them), the others `step`; every request has between `low` and `high` tokens cached already.
def _tables(name, B, chunks, chunk, step, low, high, page, padded, lengths):
    return {"name": name, "op": "tables", "B": B, "chunks": chunks, "chunk": chunk, "step": step, "low": low, "high": high,
            "page": page, "padded": padded, "lengths": lengths}


def _write(name, T, Hk, D, page, skipped):
    return {"name": name, "op": "write", "T": T, "Hk": Hk, "D": D, "page": page, "skipped": skipped}


def _attention(name, B, chunks, chunk, step, low, high, Hq, Hk, D, page, shared, lse, lengths):
    return {"name": name, "op": "attention", "B": B, "chunks": chunks, "chunk": chunk, "step": step, "low": low,
            "high": high, "Hq": Hq, "Hk": Hk, "D": D, "page": page, "shared": shared, "lse": lse, "lengths": lengths}


def listed():
    return [
        # one request being decoded
        _tables("tables B1", 1, 0, 0, 1, 700, 700, 16, 0, 1),
        # a decode batch with a piece of a prompt among it, padded to the size its graph was captured at
        _tables("tables B64 mixed", 64, 1, 449, 1, 10, 4000, 32, 30, 2),
        # many prompts at once
        _tables("tables B511 prompts", 511, 500, 31, 1, 0, 900, 16, 0, 3),
        # the key and value heads of one token being decoded
        _write("write T1", 1, 4, 128, 16, 0.0),
        # a ragged chunk, a tenth of it padding
        _write("write T777", 777, 8, 96, 32, 0.1),
        # a large prefill
        _write("write T8192", 8192, 4, 128, 64, 0.0),
        # one request being decoded: 32 query heads on 4 key heads of 128
        _attention("attention B1", 1, 0, 0, 1, 700, 700, 32, 4, 128, 16, 0, False, 1),
        # a decode batch of very different lengths
        _attention("attention B64 decode", 64, 0, 0, 1, 200, 5000, 32, 4, 128, 64, 0, False, 2),
        # four drafted tokens of every request being verified, 7 query heads to a key head
        _attention("attention B24 verify", 24, 0, 0, 4, 1000, 9000, 28, 4, 128, 32, 0, False, 3),
        # a piece of a prompt on what is cached of it, with requests being decoded; heads of 64
        _attention("attention B9 chunk", 9, 1, 501, 1, 3000, 7000, 24, 8, 64, 128, 0, True, 4),
        # a large prefill of one prompt
        _attention("attention T8192 prefill", 1, 1, 8192, 1, 0, 0, 32, 4, 128, 64, 0, False, 5),
        # requests that follow one long prompt, 8192 tokens of it in the same pages
        _attention("attention B128 shared", 128, 0, 0, 1, 8210, 8700, 32, 4, 128, 16, 8192, False, 6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "write", "attention", "attention", "attention"])
    lengths = rng.randrange(1000000)
    if op == "tables":
        B = _log(rng, 1, 1024)
        high = _log(rng, 1, 8192)
        chunks = rng.randint(0, B)
        c = _tables("", B, chunks, _log(rng, 1, max(2, 16384 // (chunks + 1))), rng.choice([1, 1, 4]), min(high, rng.choice([0, 100])),
                    high, rng.choice([16, 32, 64, 128]), rng.choice([0, 0, 17, 100]), lengths)
    elif op == "write":
        Hk, D = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 80, 96, 128, 192, 256])
        c = _write("", min(_log(rng, 1, 8192), 8192 * 512 // (Hk * D)), Hk, D, rng.choice([16, 32, 64, 128]),
                   rng.choice([0.0, 0.0, 0.2]))
    else:
        Hq, Hk, D = rng.choice([(32, 4, 128), (16, 2, 128), (28, 4, 128), (64, 8, 128), (12, 12, 64), (24, 8, 64), (20, 4, 96),
                                (40, 8, 80), (16, 16, 128)])
        page = rng.choice([16, 32, 64, 128])
        kind = rng.choice(["decode", "decode", "verify", "chunk", "prefill", "shared"])
        if kind in ("decode", "verify"):   # at most 2^18 cached tokens of 4 heads of 128
            high = _log(rng, 32, 32768)
            B = max(1, min(_log(rng, 1, 256), (1 << 27) // (high * Hk * D)))
            c = _attention("", B, 0, 0, 1 if kind == "decode" else rng.randint(2, 8), rng.choice([1, high // 4 + 1]), high, Hq, Hk,
                           D, page, 0, rng.random() < 0.25, lengths)
        elif kind == "chunk":
            chunk, high = _log(rng, 20, 1000), _log(rng, 64, 16384)
            B = max(1, min(rng.randint(1, 12), 8192 * 8192 // (chunk * (high + chunk))))
            c = _attention("", B, rng.randint(1, min(B, 3)), chunk, 1, high // 3, high, Hq, Hk, D, page, 0, rng.random() < 0.25, lengths)
        elif kind == "prefill":
            B = rng.choice([1, 1, 2, 5])
            chunk = _log(rng, 100, 8192 // B if Hq * D <= 4096 else 4096 // B)
            c = _attention("", B, B, chunk, 1, 0, 0, Hq, Hk, D, page, 0, False, lengths)
        else:
            shared, own_most = page * max(1, _log(rng, 256, 16384) // page), _log(rng, 16, 1024)
            B = max(2, min(_log(rng, 2, 256), (1 << 29) // ((shared + own_most) * Hk * D)))
            c = _attention("", B, 0, 0, rng.choice([1, 1, 1, 3]), shared, shared + own_most, Hq, Hk, D, page, shared,
                           rng.random() < 0.25, lengths)
    del c["name"]
    return c


def _lengths(case):
    """[(tokens cached, new tokens)] of the case's requests; a chunk is up to an eighth shorter than named."""
    r = random.Random(case["lengths"])
    chunks, B = case["chunks"], case["B"]
    got = []
    for b in range(B):
        low, high = case["low"], case["high"]
        cached = r.randint(low, high) if b % 4 or low == 0 else _log(r, low, high)
        n = case["chunk"]
        got.append((cached, (n if B == 1 else n - r.randint(0, n // 8)) if b < chunks else case["step"]))
    return got


# --------------------------------------------------------------------------------- their inputs
def _rand(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    page = case["page"]
    if case["op"] == "write":
        T, Hk, D = case["T"], case["Hk"], case["D"]
        pages = 2 * (T + page - 1) // page + 3
        slots = torch.randperm(pages, generator=g, device="cuda")[:, None] * page + torch.arange(page, device="cuda")
        start = int(torch.randint(0, page, (1,), generator=g, device="cuda"))   # the first page is partly filled
        slots = slots.flatten()[start:start + T]
        skip = torch.rand(T, generator=g, device="cuda") < case["skipped"]      # padding
        s["slots"] = torch.where(skip, -1, slots).to(torch.int32)
        s["k"] = _rand((T, Hk, D), g)
        s["v"] = _rand((T, 10 * Hk * D), g)[:, 9 * Hk * D:].view(T, Hk, D)      # values of merged q/k/v rows
        s["kc"], s["vc"] = _rand((pages, Hk, page, D), g), _rand((pages, Hk, page, D), g)
        if own:
            s["handle"], s["workspace"] = _the_handle(), _pkg().alloc_cache_workspace()
        return s
    lens = _lengths(case)
    B, T = len(lens), sum(n for _, n in lens)
    held = [(c + page - 1) // page for c, _ in lens]                   # pages that a request has before the step,
    need = [(c + n + page - 1) // page for c, n in lens]               # and after it
    width = max(need) + 2
    shared = case.get("shared", 0) // page
    used = shared + sum(n - shared for n in need)
    pages = used + used // 8 + 4
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    if case["op"] == "tables":
        have = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        at = torch.arange(width, device="cuda") < _ints(held)[:, None]
        have[at] = order[:sum(held)]
        s["tables"], s["free"] = have, order[sum(held):].contiguous()
        s["taken"] = torch.randint(0, 3, (1,), generator=g, device="cuda", dtype=torch.int32)
        s["cached"], s["new"] = _ints([c for c, _ in lens]), _ints([n for _, n in lens])
        s["T"] = T + case["padded"]
        if own:
            s["handle"], s["workspace"] = _the_handle(), _pkg().alloc_cache_workspace()
        return s
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    s["q"] = _rand((T, Hq, D), g)
    s["kc"], s["vc"] = _rand((pages, Hk, page, D), g), _rand((pages, Hk, page, D), g)
    tables = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(width, device="cuda") < _ints(need)[:, None]
    at[:, :shared] = False
    tables[at] = order[shared:shared + int(at.sum())]
    tables[:, :shared] = order[:shared]
    s["tables"], s["kv"] = tables, _ints([c + n for c, n in lens])
    s["offsets"] = _ints(np.cumsum([0] + [n for _, n in lens]).tolist())
    s["most"], s["longest"] = max(n for _, n in lens), max(c + n for c, n in lens)   # the program's scheduler knows both
    if own:
        s["handle"] = _the_handle()
        s["workspace"] = _pkg().alloc_attention_workspace(T, Hq, Hk, D)
    return s


# ------------------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _own_tables(s):
    o = _pkg().moe_lora_page_tables(s["handle"], s["tables"], s["cached"], s["new"], s["case"]["page"], s["free"], s["taken"], s["T"],
                                    workspace=s["workspace"])
    return s["tables"], o["kv_lens"], o["query_offsets"], o["slot_map"], o["positions"], o["taken"]


def _own_write(s):
    _pkg().moe_lora_cache_write(s["handle"], s["k"], s["v"], s["kc"], s["vc"], s["slots"], workspace=s["workspace"])
    return s["kc"], s["vc"]


def _own_attention(s):
    c = s["case"]
    one = s["most"] == 1   # a token of every request: no offsets are needed
    return _pkg().moe_lora_attention(s["handle"], s["q"], s["kc"], s["vc"], s["tables"], s["kv"],
                                     query_offsets=None if one else s["offsets"], max_query_len=s["most"],
                                     shared_len=c["shared"], return_lse=c["lse"], workspace=s["workspace"])


_run_own = {"tables": _own_tables, "write": _own_write, "attention": _own_attention}


def _plain_tables(s):
    page, tables, T = s["case"]["page"], s["tables"], s["T"]
    B = tables.shape[0]
    cached, new = s["cached"].long(), s["new"].long()
    held, need = (cached + page - 1) // page, (cached + new + page - 1) // page
    more = need - held
    first = s["taken"].long() + torch.cumsum(more, 0) - more             # of the free pages, each request's first
    col = torch.arange(tables.shape[1], device=tables.device)
    mine = (col >= held[:, None]) & (col < need[:, None])
    at = (first[:, None] + col - held[:, None]).clamp(0, s["free"].shape[0] - 1)
    tables.copy_(torch.where(mine, s["free"][at], tables))
    end = torch.cumsum(new, 0)
    t = torch.arange(T, device=tables.device)
    req = (t[:, None] >= end).sum(1)                                      # each token's request; B: padding
    real = req < B
    req = req.clamp(max=B - 1)
    pos = cached[req] + t - (end - new)[req]
    pos = torch.where(real, pos, 0)
    slot = torch.where(real, tables[req, pos // page].long() * page + pos % page, -1)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=tables.device), end])
    i = torch.int32
    return tables, (cached + new).to(i), offsets.to(i), slot.to(i), pos.to(i), s["taken"] + more.sum().to(i)


def _plain_write(s):
    page = s["case"]["page"]
    real = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][real].long()
    s["kc"][slot // page, :, slot % page] = s["k"][real]
    s["vc"][slot // page, :, slot % page] = s["v"][real]
    return s["kc"], s["vc"]


def _plain_attention(s):
    c = s["case"]
    Hk, G, D, n = c["Hk"], c["Hq"] // c["Hk"], c["D"], s["most"]
    B, width = s["tables"].shape
    T = s["q"].shape[0]
    width = min(width, (s["longest"] + c["page"] - 1) // c["page"])
    pages = s["tables"][:, :width].clamp(min=0).long()
    k = s["kc"][pages].transpose(1, 2).reshape(B, Hk, -1, D).float()
    v = s["vc"][pages].transpose(1, 2).reshape(B, Hk, -1, D).float()
    start, count = s["offsets"][:-1].long(), s["offsets"].diff().long()
    i = torch.arange(n, device=k.device)
    q = s["q"][(start[:, None] + i).clamp(max=T - 1)].float()             # [B, n, Hq, D], the rows behind `count` not used
    q = q.view(B, n, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * n, D)
    x = (q @ k.transpose(2, 3)).view(B, Hk, G, n, -1) / math.sqrt(D)
    sees = s["kv"].long()[:, None] - count[:, None] + i + 1               # keys that query i sees
    x = x.masked_fill(torch.arange(k.shape[2], device=k.device) >= sees[:, None, None, :, None], -math.inf)
    m = x.amax(4, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    x = torch.exp(x - m)
    total = x.sum(4, keepdim=True)
    o = (x.view(B, Hk, G * n, -1) @ v).view(B, Hk, G, n, D)
    o = torch.where(total > 0, o / total, 0.0)
    t = torch.arange(T, device=k.device)
    req = torch.searchsorted(s["offsets"][1:].long(), t, right=True)
    out = o.permute(0, 3, 1, 2, 4)[req, t - start[req]].reshape(T, Hk * G, D).to(torch.bfloat16)
    if not c["lse"]:
        return out
    lse = (m + torch.log(total))[..., 0].permute(0, 3, 1, 2)[req, t - start[req]].reshape(T, Hk * G)
    return out, lse


_run_plain = {"tables": _plain_tables, "write": _plain_write, "attention": _plain_attention}


# ------------------------------------------------------------------------- what a pass must cost
def work(case):
    if case["op"] == "write":
        n = round(case["T"] * (1.0 - case["skipped"]))
        return {"bytes": 8 * n * case["Hk"] * case["D"] + 4 * case["T"], "flops": 0}
    lens, page = _lengths(case), case["page"]
    T = sum(n for _, n in lens)
    if case["op"] == "tables":   # lengths in and out, slots, positions, the new pages, the pages of the new tokens
        fresh = sum((c + n + page - 1) // page - (c + page - 1) // page for c, n in lens)
        return {"bytes": 16 * len(lens) + 8 * (T + case["padded"]) + 8 * fresh + 4 * len(lens), "flops": 0}
    Hq, Hk, D, shared = case["Hq"], case["Hk"], case["D"], case["shared"]
    keys = shared + sum(c + n - shared for c, n in lens)
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in lens)
    return {"bytes": 4 * T * Hq * D + 4 * keys * Hk * D + 4 * (keys // page) + (4 * T * Hq if case["lse"] else 0),
            "flops": 4 * Hq * D * pairs}


# ---------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The definitions request by request, on the inputs of prepare(case, seed)."""
    s = prepare(case, seed)
    page = case["page"]
    if case["op"] == "write":
        kc, vc = s["kc"].double(), s["vc"].double()
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                kc[slot // page, :, slot % page] = s["k"][t].double()
                vc[slot // page, :, slot % page] = s["v"][t].double()
        return kc, vc
    if case["op"] == "tables":
        tables, free, taken = s["tables"].tolist(), s["free"].tolist(), s["taken"].item()
        kv, offsets, slots, positions = [], [0], [], []
        for row, (cached, new) in zip(tables, _lengths(case)):
            for p in range(cached, cached + new):
                if p % page == 0:   # the first token of a page
                    row[p // page] = free[taken]
                    taken += 1
                slots.append(row[p // page] * page + p % page)
                positions.append(p)
            kv.append(cached + new)
            offsets.append(offsets[-1] + new)
        slots += [-1] * case["padded"]
        positions += [0] * case["padded"]
        return _ints(tables), _ints(kv), _ints(offsets), _ints(slots), _ints(positions), _ints([taken])
    lens = _lengths(case)
    if 4 * case["Hq"] * case["D"] * sum(n * (c + n) for c, n in lens) > 5e12:
        return None
    G, D = case["Hq"] // case["Hk"], case["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    t = 0
    for row, (cached, new) in zip(s["tables"], lens):
        n = cached + new
        mine = row[:(n + page - 1) // page].long()
        hidden = torch.ones((new, n), dtype=torch.bool, device="cuda").triu(cached + 1)
        for h in range(case["Hk"]):
            k = s["kc"][mine, h].reshape(-1, D)[:n].double()
            v = s["vc"][mine, h].reshape(-1, D)[:n].double()
            for q in range(h * G, h * G + G):
                x = torch.einsum("td,nd->tn", s["q"][t:t + new, q].double(), k).mul_(D ** -0.5).masked_fill_(hidden, -math.inf)
                lse[t:t + new, q] = torch.logsumexp(x, 1)
                out[t:t + new, q] = torch.softmax(x, 1) @ v
        t += new
    return (out, lse) if case["lse"] else out
