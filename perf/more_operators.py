"""What is measured of the operators whose rows have weights of their own: route_topk (a router: the k
experts of each row, their weights, and the rows sorted by expert), w8a8_mul_mat_experts (matrix products
grouped by expert over int8 weights, ragged) and lora_add (low-rank adapters of many requests beside a
shared projection).

An item is one (row, expert) pair: item row * k + j is a row's j-th choice. A plan holds the items sorted
by owner (expert or adapter), ascending within each: start[owners + 1] and list[items].

With `own` false every operator runs in its plain form: elementary torch operations in 32 bits, in 64
where an integer sum would not fit."""

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    route = {"op": "route", "dtype": "f32", "sigmoid": False, "norm": True, "bias": False}
    experts = {"op": "experts", "dtype": "f32", "skew": 0.7}
    lora = {"op": "lora", "dtype": "f32", "none": 0.0}
    return [
        # one token's two experts of eight: latency alone
        {"name": "route one token", **route, "rows": 1, "experts": 8, "k": 2},
        # a serving step with sigmoid scores and a balancing bias, an odd number of experts, 16-bit logits
        {"name": "route odd bf16", **route, "dtype": "bf16", "rows": 1003, "experts": 60, "k": 4, "sigmoid": True,
         "bias": True},
        # a long prompt over many experts
        {"name": "route prompt", **route, "rows": 8000, "experts": 128, "k": 8},
        # one token through the gate and up projections of its two experts
        {"name": "experts one token", **experts, "rows": 1, "experts": 8, "k": 2, "N": 2 * 2048, "K": 1536,
         "form": "up"},
        # a serving step, gate and up: about four rows for each of 128 experts, weights read once
        {"name": "experts tokens up", **experts, "rows": 64, "experts": 128, "k": 8, "N": 2 * 768, "K": 2048,
         "form": "up"},
        # the same step's down projection, the experts' rows weighted and summed per token
        {"name": "experts tokens down", **experts, "rows": 64, "experts": 128, "k": 8, "N": 2048, "K": 768,
         "form": "down"},
        # a prompt, gate and up, 16-bit rows
        {"name": "experts prompt up", **experts, "dtype": "bf16", "rows": 4096, "experts": 128, "k": 8, "N": 2 * 768,
         "K": 2048, "form": "up"},
        # a shorter ragged prompt over few large experts, down projection
        {"name": "experts prompt down", **experts, "rows": 1777, "experts": 8, "k": 2, "N": 1536, "K": 8960,
         "form": "down"},
        # one token of one fine-tune
        {"name": "lora one token", **lora, "rows": 1, "adapters": 1, "rank": 16, "N": 1536, "K": 1536, "runs": 1},
        # a serving step: a token each of 64 requests over 40 fine-tunes
        {"name": "lora tokens", **lora, "rows": 64, "adapters": 40, "rank": 32, "N": 2048, "K": 2048, "runs": 64},
        # prompts of twelve requests, each with its fine-tune
        {"name": "lora prompts", **lora, "rows": 8000, "adapters": 12, "rank": 64, "N": 2048, "K": 2048, "runs": 12},
        # ragged prompts of small fine-tunes beside requests that have none, a wide projection, 16-bit rows
        {"name": "lora some rows bf16", **lora, "dtype": "bf16", "rows": 5003, "adapters": 7, "rank": 8, "N": 8960,
         "K": 1536, "runs": 23, "none": 0.3},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "experts", "lora", "lora"])
    case = {"op": op, "dtype": rng.choice(["f32", "f32", "bf16", "f16"])}
    if op == "route":
        experts = _log(rng, 4, 256)
        k = rng.randint(1, min(8, experts))
        return {**case, "rows": _log(rng, 1, 8000 * 128 // max(experts, 128)), "experts": experts, "k": k,
                "sigmoid": rng.random() < 0.3, "norm": k > 1 and rng.random() < 0.7, "bias": rng.random() < 0.3}
    if op == "experts":
        experts = rng.choice([4, 8, 16, 60, 64, 128])
        k = rng.randint(1, min(8, experts))
        form = rng.choice(["up", "down", "plain"])
        K = 16 * _log(rng, 16, 560)
        N = 32 * _log(rng, 8, 280) if form == "up" else _log(rng, 200, 8960)
        while experts * N * K > 128 * 1536 * 2048:
            N = (N // 2 + 31) // 32 * 32
            K = max(256, K // 3 * 2 // 16 * 16)
        most = max(1, 32768 * 1536 * 2048 // (N * K * k))
        return {**case, "rows": _log(rng, 1, min(4096, most)), "experts": experts, "k": k, "N": N, "K": K, "form": form,
                "skew": rng.choice([0.0, 0.5, 1.0, 2.0])}
    rank = rng.choice([8, 16, 16, 24, 32, 64, 128])
    K, N = 8 * _log(rng, 32, 1120), _log(rng, 200, 8960)
    rows = _log(rng, 1, max(1, min(8000, 8000 * 4096 // (K + 2 * N))))
    runs = rng.choice([rows, _log(rng, 1, min(rows, 64))])
    adapters = min(_log(rng, 1, 64), (64 << 20) // (rank * (K + N)) + 1)
    return {**case, "rows": rows, "adapters": adapters, "rank": rank, "N": N, "K": K, "runs": runs,
            "none": rng.choice([0.0, 0.0, 0.3])}


def _owners_in_use(case):
    """How many experts or adapters a case's rows are likely to reach (each owner alike)."""
    if case["op"] == "experts":
        n = case["experts"]
        return n * (1 - (1 - case["k"] / n) ** case["rows"])
    n = case["adapters"]
    return n * (1 - (1 - 1 / n) ** case["runs"]) if n > 1 else 1


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    rows = case["rows"]
    if case["op"] == "route":
        # logits in; ids, weights and list out, and the starts
        return {"bytes": rows * case["experts"] * size + rows * case["k"] * 12 + 4 * (case["experts"] + 1),
                "flops": 3 * rows * case["experts"]}
    N, K = case["N"], case["K"]
    if case["op"] == "experts":
        items = rows * case["k"]
        x_rows = items if case["form"] == "down" else rows
        y = {"up": items * N // 2, "down": rows * N, "plain": items * N}[case["form"]]
        return {"bytes": _owners_in_use(case) * N * (K + 4) + x_rows * K * size + y * size + items * 8,
                "flops": 2 * items * N * K}
    share, rank = 1 - case["none"], case["rank"]
    return {"bytes": share * rows * (K + 2 * N) * size + _owners_in_use(case) * rank * (K + N) * 2,
            "flops": 2 * share * rows * rank * (K + N)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, rows = DTYPES[case["dtype"]], case["rows"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    st = {"case": case}
    if case["op"] == "route":
        # a trained router's logits: some experts liked more than others
        st["logits"] = (normal(rows, case["experts"], std=1.5) + normal(case["experts"], std=0.5)).to(dtype)
        st["bias"] = normal(case["experts"], std=0.3) if case["bias"] else None
        if own:
            from int8_quantized_matmul_gb300 import i2s
            st["call"] = i2s.RouteTopk(st["logits"], case["k"], bias=st["bias"], sigmoid=case["sigmoid"],
                                       norm=case["norm"])
        return st
    N, K = case["N"], case["K"]
    if case["op"] == "experts":
        E, k = case["experts"], case["k"]
        # int8 weights as per-channel quantization leaves them
        st["wq"] = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
        for e in range(E):
            st["wq"][e] = normal(N, K, std=36.0).round_().clamp_(-127, 127)
        st["bscale"] = torch.exp(normal(E, N, std=0.3)) * (0.02 / 36)
        liked = normal(rows, E) + normal(E, std=case["skew"])
        st["expert"] = liked.topk(k).indices.to(torch.int32).contiguous()
        st["weight"] = torch.softmax(normal(rows, k), -1)
        x_rows = rows * k if case["form"] == "down" else rows
        x = normal(x_rows, K)
        if case["form"] == "down":  # the product of a gate and an up value
            x *= torch.nn.functional.silu(normal(x_rows, K))
        st["x"] = (x * torch.exp(normal(K, std=0.3))).to(dtype)
        out = {"up": (rows * k, N // 2), "down": (rows, N), "plain": (rows * k, N)}[case["form"]]
        st["out"] = torch.zeros(out, dtype=dtype, device="cuda")
        if own:
            from int8_quantized_matmul_gb300 import i2s
            plan = i2s.route_plan(st["expert"].view(-1), E)
            st["call"] = i2s.W8A8Experts(st["wq"], st["bscale"], plan, st["x"], out=st["out"],
                                         x_group=1 if case["form"] == "down" else k, swiglu=case["form"] == "up",
                                         weight=st["weight"] if case["form"] == "down" else None)
        return st
    adapters, rank = case["adapters"], case["rank"]
    half = torch.float16 if dtype == torch.float16 else torch.bfloat16
    st["A"] = normal(adapters, rank, K, std=K ** -0.5).to(half)
    st["B"] = normal(adapters, N, rank, std=0.05).to(half)
    st["scale"] = torch.exp(normal(adapters, std=0.3))
    # runs of neighbouring rows (the tokens of a request) share an adapter, or have none
    runs = case["runs"]
    run = torch.zeros(rows, dtype=torch.int64, device="cuda")
    run[1 + torch.randperm(rows - 1, generator=gen, device="cuda")[:runs - 1]] = 1
    owner = torch.randint(0, adapters, (runs,), generator=gen, device="cuda")
    owner = torch.where(torch.rand(runs, generator=gen, device="cuda") < case["none"], -1, owner)
    owner[:1].clamp_(min=0)  # one run at least has an adapter
    st["owner"] = owner[run.cumsum(0)].to(torch.int32)
    st["x"] = (normal(rows, K) * torch.exp(normal(K, std=0.3))).to(dtype)
    st["base"] = normal(rows, N).to(dtype)
    st["out"] = torch.zeros((rows, N), dtype=dtype, device="cuda")
    if own:
        from int8_quantized_matmul_gb300 import i2s
        plan = i2s.route_plan(st["owner"], adapters)
        st["call"] = i2s.LoraAdd(st["A"], st["B"], plan, st["x"], st["base"], out=st["out"], scale=st["scale"])
    return st


def run(st):
    op = st["case"]["op"]
    if op == "route":
        if own:
            call = st["call"]
            call()
            return {"expert": call.expert, "weight": call.weight, "start": call.plan.start, "list": call.plan.list}
        return _plain_route(st)
    if own:
        st["call"]()
        return st["out"]
    return _plain_experts(st) if op == "experts" else _plain_lora(st)


# -- the plain forms ------------------------------------------------------------------------------

def _plain_plan(owner, owners):
    """start and list of the items sorted by owner, in order within each."""
    order = (owner.long() * owner.numel() + torch.arange(owner.numel(), device="cuda")).argsort()
    count = (owner[:, None] == torch.arange(owners, device="cuda")).sum(0)
    start = torch.nn.functional.pad(count.cumsum(0), (1, 0))
    return start.to(torch.int32), order.to(torch.int32)


def _plain_route(st):
    case = st["case"]
    logit = st["logits"].float()
    score = logit + st["bias"] if case["bias"] else logit.clone()
    index = torch.arange(case["experts"], device="cuda")
    chosen = []
    for _ in range(case["k"]):
        top = score.amax(1, keepdim=True)
        best = torch.where(score == top, index, case["experts"]).amin(1, keepdim=True)
        chosen.append(best)
        score = score.masked_fill(index == best, -math.inf)
    chosen = torch.cat(chosen, 1)
    value = logit.gather(1, chosen)
    if case["sigmoid"]:
        weight = 1 / (1 + torch.exp(-value))
        if case["norm"]:
            weight = weight / weight.sum(1, keepdim=True)
    else:
        base = value if case["norm"] else logit
        top = base.amax(1, keepdim=True)
        weight = torch.exp(value - top) / torch.exp(base - top).sum(1, keepdim=True)
    start, order = _plain_plan(chosen.view(-1), case["experts"])
    return {"expert": chosen.to(torch.int32), "weight": weight, "start": start, "list": order}


def _codes(x):
    """int8 codes (as floats) and the scale of each row, binary32 step by step."""
    x = x.float()
    amax = x.abs().amax(1, keepdim=True).clamp_min(1e-9)
    unit = torch.full_like(amax, 127.0)  # divided by a tensor: a number's reciprocal would be multiplied
    step = (x * (unit / amax)).clamp_(-127, 127)
    whole = step.trunc()
    return whole + torch.where((step - whole).abs() >= 0.5, step.sign(), 0.0), amax / unit


def _plain_experts(st):
    case = st["case"]
    k, form = case["k"], case["form"]
    code, scale = _codes(st["x"])
    # two digits: sums of their products with a weight stay below 2^24, whole numbers in 32 bits
    high = (code * 0.0625 + 0.5).floor()
    low = code - 16 * high
    expert = st["expert"].view(-1)
    d = torch.zeros((expert.numel(), case["N"]), device="cuda")
    for e in range(case["experts"]):
        item = (expert == e).nonzero()[:, 0]
        row = item if form == "down" else item // k
        w = st["wq"][e].float().T
        dot = (high[row] @ w).double() * 16 + (low[row] @ w).double()
        d[item] = (scale[row] * st["bscale"][e]) * dot.float()
    if form == "up":
        gate, up = d.chunk(2, 1)
        d = gate / (1 + torch.exp(-gate)) * up
    if form == "down":
        d = (d.view(case["rows"], k, -1) * st["weight"][:, :, None]).sum(1)
    return d.to(st["x"].dtype)


def _plain_lora(st):
    out = torch.zeros_like(st["base"])
    for a in range(st["case"]["adapters"]):
        row = (st["owner"] == a).nonzero()[:, 0]
        inner = st["x"][row].float() @ st["A"][a].float().T
        delta = (inner @ st["B"][a].float().T) * st["scale"][a]
        out[row] = (st["base"][row].float() + delta).to(out.dtype)
    return out


# -- the definitions in 64 bits --------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        logit = st["logits"].double().cpu()
        # the score is a binary32 sum by definition
        score = (logit + st["bias"].double().cpu()).float().double() if case["bias"] else logit
        chosen = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :case["k"]]
        value = torch.gather(logit, 1, chosen)
        if case["sigmoid"]:
            weight = torch.sigmoid(value)
            weight = weight / weight.sum(1, keepdim=True) if case["norm"] else weight
        elif case["norm"]:
            weight = torch.softmax(value, 1)
        else:
            weight = torch.gather(torch.softmax(logit, 1), 1, chosen)
        flat = chosen.reshape(-1)
        start = [0]
        for n in torch.bincount(flat, minlength=case["experts"]).tolist():
            start.append(start[-1] + n)
        return {"expert": chosen.to(torch.int32).cuda(), "weight": weight.cuda(),
                "start": torch.tensor(start, dtype=torch.int32, device="cuda"),
                "list": torch.sort(flat, stable=True).indices.to(torch.int32).cuda()}
    if case["op"] == "experts":
        x = st["x"].double()
        # the codes are defined by binary32 steps: each rounded to it here, too
        amax = x.abs().amax(1).clamp_min(float(torch.tensor(1e-9)))
        factor = (127 / amax).float().double()
        code = (x * factor[:, None]).float().double().clamp(-127, 127)
        code = code.sign() * (code.abs() + 0.5).floor()
        scale = (amax / 127).float().double()
        k, form = case["k"], case["form"]
        flat = st["expert"].view(-1).long()
        order = torch.sort(flat, stable=True).indices
        d = torch.empty((flat.numel(), case["N"]), dtype=torch.float64, device="cuda")
        for part in torch.split(order, torch.bincount(flat, minlength=case["experts"]).tolist()):
            if part.numel() == 0:
                continue
            e = flat[part[0]]
            row = part if form == "down" else torch.div(part, k, rounding_mode="floor")
            d[part] = torch.einsum("rk,nk->rn", code[row], st["wq"][e].double()) * scale[row, None] * \
                st["bscale"][e].double()
        if form == "up":
            half = case["N"] // 2
            return torch.nn.functional.silu(d[:, :half]) * d[:, half:]
        if form == "down":
            return torch.einsum("tkn,tk->tn", d.unflatten(0, (-1, k)), st["weight"].double())
        return d
    owner = st["owner"].long()
    here = owner >= 0
    result = torch.zeros(st["base"].shape, dtype=torch.float64, device="cuda")
    for a in owner[here].unique().tolist():
        row = owner == a
        both = st["B"][a].double() @ (st["A"][a].double() @ st["x"][row].double().T)
        result[row] = st["base"][row].double() + both.T * st["scale"][a].double()
    return result
