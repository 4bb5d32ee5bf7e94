"""The operators around the routed expert layer, as cases to measure.

Three operators stand between the residual stream and the expert layer of a model served with many
LoRA adapters at once:

  linear   a shared projection with per-token adapters beside it (moe_lora_linear)
  select   the choice of experts from the router's logits (moe_lora_select_experts)
  rope     the norm of every query and key head with the position rotation (moe_lora_qk_norm_rope)

Where `own` is false `run` computes them from elementary torch operations in 32 bits; where it is
true it calls the framework.  `exact` computes them in 64 bits.
"""
import math

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
def _linear(name, T, K, N, ranks, scalings, spread, out, bias=False):
    return {"name": name, "op": "linear", "T": T, "K": K, "N": N, "ranks": ranks, "scalings": scalings,
            "spread": spread, "out": out, "bias": bias}


def _select(name, T, E, k, score, logits, bias, n_group, topk_group, group, renormalize, factor, masked):
    return {"name": name, "op": "select", "T": T, "E": E, "k": k, "score": score, "logits": logits, "bias": bias,
            "n_group": n_group, "topk_group": topk_group, "group": group, "renormalize": renormalize,
            "factor": factor, "masked": masked}


def _rope(name, T, Hq, Hk, D, R, weight, interleaved, most):
    return {"name": name, "op": "rope", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "weight": weight,
            "interleaved": interleaved, "most": most}


def listed():
    return [
        # one request being decoded: the output projection of a 2048-wide model, one rank-16 adapter
        _linear("linear T1", 1, 2048, 2048, "16", "2.0", "mixed", "bf16"),
        # a decode batch of the multi-adapter configuration: merged q/k/v rows, four resident adapters
        _linear("linear T64 four adapters", 64, 2048, 5120, "8,16,32,64", "2.0,1.0,0.5,0.25", "mixed", "bf16"),
        # the router's own projection of the 384-expert configuration at its decode batch: float32
        # logits, no adapter
        _linear("linear T128 router", 128, 7168, 384, "", "", "mixed", "fp32", bias=True),
        # a ragged chunk of prompts: the gate and up rows of a shared expert (2 x 768), odd token count
        _linear("linear T777 ragged", 777, 2048, 1536, "16,16,12", "1.0,2.0,0.5", "runs", "bf16"),
        # a large prefill of the 7168-wide configuration, the prompts of four adapters one after another
        _linear("linear T8192 prefill", 8192, 7168, 4096, "16,32,16,64", "2.0,1.0,0.5,0.25", "runs", "bf16"),
        # one token being decoded: sigmoid scores, a balance bias, 8 groups of which 4 stay
        _select("select T1 grouped", 1, 256, 8, "sigmoid", "fp32", True, 8, 4, "top2", True, 2.5, 0.0),
        # the decode configuration's routing: softmax over 128 experts, bf16 logits
        _select("select T64 softmax", 64, 128, 8, "softmax", "bf16", False, 1, 1, "max", True, 1.0, 0.0),
        # the 384-expert configuration's prefill, an odd number of tokens, some experts masked out
        _select("select T4095 bias", 4095, 384, 8, "sigmoid", "bf16", True, 1, 1, "max", True, 2.827, 0.02),
        # a large prefill with grouped softmax routing, weights not renormalised
        _select("select T16384 grouped", 16384, 256, 6, "softmax", "fp32", False, 8, 3, "max", False, 16.0, 0.0),
        # one token being decoded: 32 query and 4 key heads of 128
        _rope("rope T1", 1, 32, 4, 128, 128, "bf16", False, 40960),
        # an odd chunk, partly rotated heads in neighbouring pairs
        _rope("rope T333 partial", 333, 24, 8, 192, 64, "fp32", True, 131072),
        # a large prefill
        _rope("rope T8192", 8192, 32, 4, 128, 128, "bf16", False, 40960),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "select", "rope"])
    if op == "linear":
        T, K, N = _log(rng, 1, 8192), 8 * _log(rng, 16, 896), _log(rng, 64, 8192)
        while T * K * N > 8192 * 7168 * 4096:
            T = max(1, T // 2)
        S = rng.choice([0, 1, 2, 4, 7, 16])
        ranks = [rng.choice([4, 8, 12, 16, 32, 64]) for _ in range(S)]
        scal = [rng.choice([0.25, 0.5, 1.0, 2.0]) for _ in range(S)]
        c = _linear("", T, K, N, ",".join(map(str, ranks)), ",".join(map(str, scal)), rng.choice(["mixed", "runs"]),
                    rng.choice(["bf16", "bf16", "fp32"]), rng.choice([False, True]))
    elif op == "select":
        n_group = rng.choice([1, 1, 4, 8, 16])
        E = n_group * rng.randint(max(2, 32 // n_group), 512 // n_group)
        topk_group = rng.randint(max(1, n_group // 2), n_group)
        k = rng.randint(1, min(10, topk_group * (E // n_group)))
        c = _select("", _log(rng, 1, 16384), E, k, rng.choice(["softmax", "sigmoid"]), rng.choice(["bf16", "fp32"]),
                    rng.choice([False, True]), n_group, topk_group, rng.choice(["max", "top2"]),
                    rng.choice([False, True]), rng.choice([1.0, 2.5, 2.827]), rng.choice([0.0, 0.0, 0.05]))
    else:
        D = rng.choice([64, 80, 96, 128, 192, 256])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 7, 8])
        R = rng.choice([D, D, D // 2 // 8 * 8])
        T = min(_log(rng, 1, 8192), 8192 * 36 * 128 // ((Hq + Hk) * D))
        c = _rope("", T, Hq, Hk, D, R, rng.choice(["bf16", "fp32"]), rng.choice([False, False, True]),
                  rng.choice([8192, 40960, 131072]))
    del c["name"]
    return c


# --------------------------------------------------------------------------------- their inputs
def _ranks(case):
    return [int(r) for r in case["ranks"].split(",") if r]


def _scalings(case):
    return [float(s) for s in case["scalings"].split(",") if s]


def _slots(case, g, S):
    """Each token's adapter: drawn for every token (decode) or one prompt after another (runs)."""
    T = case["T"]
    if case["spread"] == "mixed":
        slots = torch.randint(0, S, (T,), generator=g, device="cuda")
    else:
        at = torch.rand(T, generator=g, device="cuda") < 1.0 / 300.0
        run = torch.cumsum(at.to(torch.int64), 0)
        slots = torch.randint(0, S, (T + 1,), generator=g, device="cuda")[run]
    none = torch.rand(T, generator=g, device="cuda") < 0.1
    return torch.where(none & (T > 1), -1, slots).to(torch.int32)


def _rand(shape, std, g, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T = case["T"]
    s = {"case": case}
    if case["op"] == "linear":
        K, N, ranks = case["K"], case["N"], _ranks(case)
        S, R = len(ranks), max(ranks, default=0)
        s["x"] = _rand((T, K), 1.0, g, torch.bfloat16)
        s["w"] = _rand((N, K), 1.0 / math.sqrt(K), g, torch.bfloat16)
        s["bias"] = _rand((N,), 0.1, g, torch.float32) if case["bias"] else None
        if S:
            s["A"] = _rand((S, R, K), 1.0 / math.sqrt(K), g, torch.bfloat16)
            s["B"] = _rand((S, N, R), 0.02, g, torch.bfloat16)
            s["slots"] = _slots(case, g, S)
            s["ranks"] = torch.tensor(ranks, device="cuda")
            s["scalings"] = torch.tensor(_scalings(case), device="cuda")
        if own:   # what a serving program keeps: the handle, the loaded adapters, a workspace
            pkg = _pkg()
            s["handle"] = _the_handle()
            s["adapters"] = pkg.moe_lora_linear_adapters(s["handle"], s["A"], s["B"], ranks, _scalings(case)) if S else None
            s["workspace"] = pkg.alloc_linear_workspace(T, s["adapters"])
    elif case["op"] == "select":
        E = case["E"]
        z = torch.randn((T, E), generator=g, device="cuda") * 1.5
        if case["masked"]:   # experts that the caller rules out for a token
            z = z.masked_fill(torch.rand((T, E), generator=g, device="cuda") < case["masked"], -math.inf)
        s["z"] = z.to(torch.bfloat16 if case["logits"] == "bf16" else torch.float32)
        s["bias"] = _rand((E,), 0.1 if case["score"] == "sigmoid" else 0.005, g, torch.float32) if case["bias"] else None
        if own:
            s["handle"] = _the_handle()
    else:
        Hq, Hk, D, R = case["Hq"], case["Hk"], case["D"], case["R"]
        qkv = _rand((T, (Hq + 2 * Hk) * D), 1.0, g, torch.bfloat16)   # merged rows: queries, keys, values
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        wt = torch.bfloat16 if case["weight"] == "bf16" else torch.float32
        s["wq"] = (1.0 + _rand((D,), 0.1, g, torch.float32)).to(wt)
        s["wk"] = (1.0 + _rand((D,), 0.1, g, torch.float32)).to(wt)
        freq = 1e6 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        angle = torch.arange(case["most"], device="cuda", dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)   # [most, R]
        start = int(torch.randint(0, case["most"] - T, (1,), generator=g, device="cuda"))
        s["positions"] = torch.arange(start, start + T, device="cuda", dtype=torch.int32)
        if own:
            pkg = _pkg()
            s["handle"] = _the_handle()
            s["workspace"] = pkg.alloc_qk_norm_rope_workspace()
    return s


# ------------------------------------------------------------------------------------- one pass
def run(state):
    return (_run_own if own else _run_plain)[state["case"]["op"]](state)


def _own_linear(s):
    out = torch.float32 if s["case"]["out"] == "fp32" else torch.bfloat16
    return _pkg().moe_lora_linear(s["handle"], s["x"], s["w"], adapters=s["adapters"], slot_idx=s.get("slots"),
                                  bias=s["bias"], out_dtype=out, workspace=s["workspace"])


def _own_select(s):
    pkg, c = _pkg(), s["case"]
    o = pkg.moe_lora_select_experts(
        s["handle"], s["z"], c["k"], scoring=pkg.SCORE_SIGMOID if c["score"] == "sigmoid" else pkg.SCORE_SOFTMAX,
        bias=s["bias"], n_group=c["n_group"], topk_group=c["topk_group"],
        group_score=pkg.GROUP_TOP2 if c["group"] == "top2" else pkg.GROUP_MAX, renormalize=c["renormalize"],
        routed_scaling_factor=c["factor"])
    return o["topk_ids"], o["topk_weights"]


def _own_rope(s):
    return _pkg().moe_lora_qk_norm_rope(s["handle"], s["q"], s["k"], s["wq"], s["wk"], s["table"], s["positions"],
                                        eps=1e-6, interleaved=s["case"]["interleaved"], workspace=s["workspace"])


_run_own = {"linear": _own_linear, "select": _own_select, "rope": _own_rope}


def _plain_linear(s):
    x = s["x"].float()
    y = x @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if "A" in s:
        S, R, K = s["A"].shape
        u = (x @ s["A"].float().reshape(S * R, K).t()).reshape(-1, S, R)
        slot = torch.arange(S, device=x.device)
        mine = (s["slots"][:, None] == slot)[:, :, None] & (torch.arange(R, device=x.device) < s["ranks"][:, None])
        u = torch.where(mine, u * s["scalings"][:, None], 0.0)
        y = y + u.reshape(-1, S * R) @ s["B"].float().transpose(1, 2).reshape(S * R, -1)
    return y if s["case"]["out"] == "fp32" else y.to(torch.bfloat16)


def _plain_select(s):
    c, z = s["case"], s["z"].float()
    T, E = z.shape
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-z))
    else:   # the sum is taken in 64 bits, so that it is the same in any order
        e = torch.exp(z - z.amax(1, keepdim=True))
        score = e / e.double().sum(1, keepdim=True).float()
    key = score if s["bias"] is None else score + s["bias"]
    key = torch.where(z == -math.inf, -math.inf, key)   # a masked expert is never chosen
    G = c["n_group"]
    if G > 1:
        best = key.reshape(T, G, E // G).sort(2, descending=True).values
        group = best[:, :, 0] + best[:, :, 1] if c["group"] == "top2" else best[:, :, 0]
        order = group.sort(dim=1, descending=True, stable=True).indices   # ties: the lower group
        stay = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, order[:, :c["topk_group"]], True)
        key = torch.where(stay.repeat_interleave(E // G, 1), key, -math.inf)
    picked = key.sort(dim=1, descending=True, stable=True)   # ties: the lower expert
    ids = picked.indices[:, :c["k"]]
    w = torch.where(picked.values[:, :c["k"]] > -math.inf, score.gather(1, ids), 0.0)
    if c["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids.to(torch.int32), w * c["factor"]


def _plain_rope_one(x, w, cos, sin, case):
    R = case["R"]
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + 1e-6) * w.float()
    r, rest = x[:, :, :R], x[:, :, R:]
    if case["interleaved"]:
        a, b = r[:, :, 0::2], r[:, :, 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], 3).flatten(2)
    else:
        a, b = r[:, :, :R // 2], r[:, :, R // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], 2)
    return torch.cat([r, rest], 2).to(torch.bfloat16)


def _plain_rope(s):
    c = s["case"]
    row = s["table"][s["positions"].long()][:, None]
    cos, sin = row[:, :, :c["R"] // 2], row[:, :, c["R"] // 2:]
    return _plain_rope_one(s["q"], s["wq"], cos, sin, c), _plain_rope_one(s["k"], s["wk"], cos, sin, c)


_run_plain = {"linear": _plain_linear, "select": _plain_select, "rope": _plain_rope}


# ------------------------------------------------------------------------- what a pass must cost
def work(case):
    T = case["T"]
    if case["op"] == "linear":
        K, N, r = case["K"], case["N"], _ranks(case)
        mean = 0.9 * sum(r) / len(r) if r else 0.0   # a token's rank, a tenth of the tokens without
        size = 4 if case["out"] == "fp32" else 2
        present = sum(r) if case["spread"] == "runs" or T >= len(r) else mean * T
        return {"bytes": 2 * N * K + 2 * T * K + size * T * N + 2 * present * (K + N) + (4 * T if r else 0)
                + (4 * N if case["bias"] else 0),
                "flops": 2 * T * N * K + 2 * T * mean * (K + N)}
    if case["op"] == "select":
        E = case["E"]
        return {"bytes": T * E * (2 if case["logits"] == "bf16" else 4) + (4 * E if case["bias"] else 0)
                + 8 * T * case["k"], "flops": 4 * T * E}
    H, D = case["Hq"] + case["Hk"], case["D"]
    return {"bytes": 4 * T * H * D + 4 * T * case["R"] + 4 * T + 2 * D * (2 if case["weight"] == "bf16" else 4),
            "flops": 7 * T * H * D}


# ---------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The definitions in 64 bits, on the inputs of prepare(case, seed)."""
    s = prepare(case, seed)
    if case["op"] == "linear":
        x = s["x"].double()
        y = x @ s["w"].double().T
        if s["bias"] is not None:
            y += s["bias"].double()
        for i, (r, f) in enumerate(zip(_ranks(case), _scalings(case))):
            rows = (s["slots"] == i).nonzero()[:, 0]
            y[rows] += f * (x[rows] @ s["A"][i, :r].double().T) @ s["B"][i, :, :r].double().T
        return y
    if case["op"] == "select":
        z = s["z"].double()
        masked = z == -math.inf
        p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, 1)
        key = (p + s["bias"].double() if s["bias"] is not None else p).masked_fill(masked, -math.inf)
        G, E = case["n_group"], case["E"]
        if G > 1:
            rank = key.view(-1, G, E // G).topk(2 if case["group"] == "top2" else 1, 2).values.sum(2)
            order = torch.argsort(rank, dim=1, descending=True, stable=True)
            out = torch.ones_like(rank, dtype=torch.bool)
            out[torch.arange(case["T"], device=z.device)[:, None], order[:, :case["topk_group"]]] = False
            key = key.view(-1, G, E // G).masked_fill(out[:, :, None], -math.inf).view(-1, E)
        ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :case["k"]]
        w = p.gather(1, ids) * (key.gather(1, ids) > -math.inf)
        if case["renormalize"]:
            w = torch.nan_to_num(w / w.sum(1, keepdim=True))
        return None, w * case["factor"]
    angle = s["table"].double()[s["positions"].long()]
    turn = torch.complex(angle[:, :case["R"] // 2], angle[:, case["R"] // 2:])[:, None]
    got = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.double()
        n = x / torch.sqrt(x.square().mean(2, keepdim=True) + 1e-6) * w.double()
        r = n[:, :, :case["R"]]
        pair = r.unflatten(2, (-1, 2)) if case["interleaved"] else r.unflatten(2, (2, -1)).transpose(2, 3)
        pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        r = pair.flatten(2) if case["interleaved"] else pair.transpose(2, 3).flatten(2)
        got.append(torch.cat([r, n[:, :, case["R"]:]], 2))
    return tuple(got)
