"""What is measured of the 8-bit cache operators: kv8_norm_rope (norms of queries and keys with the
position rotation), kv8_write and kv8_read (the cache quantized as it is written, and read back) and
kv8_attention (attention over it).

A cache is a pool of pages of `page` tokens. A page holds, for each KV head, a slab of the K codes
(page x dim int8), the V codes, one F32 scale for each 16 tokens of K, the same for V, and padding
to a multiple of 32 bytes. Row i of the n rows that a sequence of length `len` brings is its
position len - n + i.

With `own` false every operator runs in its plain form: elementary torch operations in 32 bits."""

import math
import random

import torch

own = False

BLOCK = 16
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    attend = {"op": "attend", "dtype": "f32", "dim": 128, "page": 64, "window": 0, "mix": 1}
    cache = {"op": "cache", "dtype": "f32", "dim": 128, "page": 64, "mix": 2}
    rope = {"op": "rope", "dtype": "f32", "dim": 128, "rot": 128, "norm": True, "pairs": "half", "fused": True}
    return [
        # one token of one short conversation: 12 query heads over 2, latency alone
        {"name": "attend one token", **attend, "q_heads": 12, "kv_heads": 2, "seqs": 1, "len_lo": 75, "len_hi": 75,
         "new_lo": 1, "new_hi": 1},
        # a serving step: 64 conversations of mixed length, one token each, 16 query heads over 8
        {"name": "attend batch of tokens", **attend, "q_heads": 16, "kv_heads": 8, "seqs": 64, "len_lo": 500,
         "len_hi": 4100, "new_lo": 1, "new_hi": 1},
        # one token over one long document, 16-bit rows
        {"name": "attend long document", **attend, "dtype": "bf16", "q_heads": 12, "kv_heads": 2, "seqs": 1,
         "len_lo": 131001, "len_hi": 131001, "new_lo": 1, "new_hi": 1},
        # drafted tokens checked in one step: 1 to 6 tokens for each of 16 sequences, small pages, a window
        {"name": "attend drafts", **attend, "q_heads": 12, "kv_heads": 2, "seqs": 16, "page": 16, "window": 2048,
         "len_lo": 900, "len_hi": 9000, "new_lo": 1, "new_hi": 6},
        # a prompt of the length that the prefill leg runs, from nothing
        {"name": "attend prompt 512", **attend, "q_heads": 12, "kv_heads": 2, "seqs": 1, "len_lo": 512, "len_hi": 512,
         "new_lo": 512, "new_hi": 512},
        # a long prompt
        {"name": "attend prompt 8000", **attend, "q_heads": 16, "kv_heads": 8, "seqs": 1, "len_lo": 8000,
         "len_hi": 8000, "new_lo": 8000, "new_hi": 8000},
        # chunks of prompts behind tokens already cached, ragged, 16-bit rows
        {"name": "attend chunks bf16", **attend, "dtype": "bf16", "q_heads": 16, "kv_heads": 8, "seqs": 5,
         "len_lo": 2100, "len_hi": 5000, "new_lo": 300, "new_hi": 2047},
        # the tokens of one serving step appended, each into a block that may hold others, and read back
        {"name": "cache append", **cache, "kv_heads": 8, "seqs": 64, "len_lo": 500, "len_hi": 4100, "new_lo": 1,
         "new_hi": 1},
        # prompts written at once and read back, 16-bit rows
        {"name": "cache prompts bf16", **cache, "dtype": "bf16", "kv_heads": 8, "seqs": 6, "len_lo": 1501,
         "len_hi": 4097, "new_lo": 1500, "new_hi": 1501},
        # queries and keys of one serving step, at far positions
        {"name": "rope tokens", **rope, "q_heads": 12, "kv_heads": 2, "rows": 8, "far": 1000000},
        # a long prompt's, as the fused projection lays them out (queries, keys and values in one row)
        {"name": "rope prompt", **rope, "q_heads": 16, "kv_heads": 8, "rows": 8000, "far": 8000},
        # part of each head rotated, neighbouring pairs, no norm, 16-bit rows
        {"name": "rope partial bf16", **rope, "dtype": "bf16", "q_heads": 32, "kv_heads": 4, "rows": 5003, "rot": 64,
         "norm": False, "pairs": "next", "fused": False, "far": 131072},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "cache", "rope"])
    case = {"op": op, "dtype": rng.choice(["f32", "f32", "bf16", "f16"]), "dim": rng.choice([64, 128, 128])}
    kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 4, 5, 6, 7, 8, 16])
    if op == "rope":
        rows = min(_log(rng, 1, 8000), 8000 * 24 * 128 // ((kv + kv * group) * case["dim"]))
        return {**case, "q_heads": kv * group, "kv_heads": kv, "rows": rows, "rot": rng.choice([case["dim"], 32]),
                "norm": rng.random() < 0.7, "pairs": rng.choice(["half", "next"]), "fused": rng.random() < 0.5,
                "far": _log(rng, rows, 2000000)}
    case |= {"page": rng.choice([16, 32, 64, 128, 256]), "mix": rng.randrange(1 << 20), "kv_heads": kv}
    if op == "cache":
        seqs = _log(rng, 1, 100)
        new = min(_log(rng, 1, 6000), 12000 // seqs + 1)
        return {**case, "seqs": seqs, "new_lo": max(1, new // 3), "new_hi": new, "len_lo": new,
                "len_hi": new + _log(rng, 1, 3000)}
    case |= {"q_heads": kv * group, "window": rng.choice([0, 0, 0, _log(rng, 16, 5000)])}
    if rng.random() < 0.55:  # a serving step, or drafts
        seqs = _log(rng, 1, 100)
        new = rng.choice([1, 1, 1, rng.randrange(2, 9)])
        most = min(131000, max(64, (200 << 20) // (seqs * kv * case["dim"]), new))
        high = max(new, _log(rng, 16, min(most, (1 << 28) // (seqs * new * kv * group))))
        return {**case, "seqs": seqs, "new_lo": 1, "new_hi": new, "len_hi": high,
                "len_lo": max(new, rng.choice([1, 2, 8]) * high // 8)}
    seqs = _log(rng, 1, 12)
    new = _log(rng, 9, 3000)
    high = _log(rng, new, 6000)
    while seqs * new * high * kv * group > 5 << 26:
        seqs, new, high = (seqs + 1) // 2, max(9, new * 3 // 4), max(9, new * 3 // 4, high * 3 // 4)
    return {**case, "seqs": seqs, "new_lo": max(1, new // 2), "new_hi": new, "len_lo": new, "len_hi": high}


def _lengths(case):
    """(cached length, new rows) of each sequence: the same for every seed."""
    rng = random.Random(case["mix"])
    return [(rng.randint(case["len_lo"], case["len_hi"]), rng.randint(case["new_lo"], case["new_hi"]))
            for _ in range(case["seqs"])]


def _slab(dim, page):
    return 2 * page * dim + (page // BLOCK * 8 + 31) // 32 * 32


def work(case):
    dim, size = case["dim"], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        values = case["rows"] * (case["q_heads"] + case["kv_heads"]) * dim
        # read and written once; the norm's square sum, its two products and the rotation
        return {"bytes": 2 * size * values, "flops": (4 if case["norm"] else 0) * values + 3 * values}
    kv, token = case["kv_heads"], 2 * dim + 8 / BLOCK
    if case["op"] == "cache":
        moved = flops = 0
        for length, new in _lengths(case):
            blocks = (length - 1) // BLOCK - (length - new) // BLOCK + 1
            held = min(length, new + BLOCK - 1)
            moved += kv * (2 * dim * size * (new + held) + token * (new + held) + token * ((length - new) % BLOCK))
            flops += kv * 2 * dim * (3 * new + held) + blocks
        return {"bytes": moved, "flops": flops}
    pairs = keys = rows = 0
    for length, new in _lengths(case):
        seen = [min(length - new + i + 1, case["window"] or length) for i in (0, new - 1)]
        first = max(0, length - new + 1 - case["window"]) if case["window"] else 0
        if case["window"]:
            pairs += sum(min(length - new + i + 1, case["window"]) for i in range(new))
        else:
            pairs += (seen[0] + seen[1]) * new // 2
        keys, rows = keys + length - first, rows + new
    return {"bytes": keys * kv * token + 2 * size * rows * case["q_heads"] * dim + 4 * rows * case["q_heads"],
            "flops": 4 * dim * pairs * case["q_heads"]}


def _turns(rot, base=1000000.0):
    """The rotation of pair i for each position, base^(-2i/rot) radians, in 2^-64 turns."""
    return torch.tensor([int(base ** (-2 * i / rot) / (2 * math.pi) * 2.0 ** 64) for i in range(rot // 2)],
                        dtype=torch.int64, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, dim, kv = DTYPES[case["dtype"]], case["dim"], case["kv_heads"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    if case["op"] == "rope":
        rows, q_heads = case["rows"], case["q_heads"]
        heads = q_heads + kv * (2 if case["fused"] else 1)
        # activations of a projection have channels of their own size
        x = (normal(rows, heads, dim) * torch.exp(normal(heads, dim, std=0.5))).to(dtype)
        q, k = x[:, :q_heads], x[:, q_heads:q_heads + kv]
        if not case["fused"]:
            q, k = q.contiguous(), k.contiguous()
        st = {"case": case, "q": q, "k": k, "turns": _turns(case["rot"]),
              "positions": torch.randint(0, case["far"] + 1, (rows,), generator=gen, device="cuda", dtype=torch.int32),
              "q_out": torch.empty((rows, q_heads, dim), dtype=dtype, device="cuda"),
              "k_out": torch.empty((rows, kv, dim), dtype=dtype, device="cuda"), "gamma_q": None, "gamma_k": None}
        if case["norm"]:
            st |= {"gamma_q": 1 + normal(dim, std=0.2), "gamma_k": 1 + normal(dim, std=0.2)}
        if own:
            from int8_quantized_matmul_gb300 import i2s
            st["call"] = i2s.Kv8NormRope(st["q"], st["k"], st["positions"], st["turns"], gamma_q=st["gamma_q"],
                                         gamma_k=st["gamma_k"], eps=1e-6, interleaved=case["pairs"] == "next",
                                         q_out=st["q_out"], k_out=st["k_out"])
        return st

    page, lengths = case["page"], _lengths(case)
    width = -(-max(length for length, _ in lengths) // page)
    used = [-(-length // page) for length, _ in lengths]
    n_pages = sum(used) + 3
    slab = _slab(dim, page)
    # a pool in use: codes as quantization leaves them, pages handed out in no order
    pool = torch.empty((n_pages, kv, slab), dtype=torch.uint8, device="cuda")
    codes = pool.view(torch.int8)[:, :, :2 * page * dim]
    for p in range(0, n_pages, 4096):
        part = codes[p:p + 4096]
        part.copy_(normal(*part.shape, std=40.0).round_().clamp_(-127, 127))
    pool.view(torch.float32)[:, :, 2 * page * dim // 4:] = torch.exp(
        normal(n_pages, kv, (slab - 2 * page * dim) // 4, std=0.3)) * 0.02
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = order[at:at + n]
        at += n
    news = [new for _, new in lengths]
    starts = [sum(news[:s]) for s in range(len(news) + 1)]
    st = {"case": case, "pool": pool.view(n_pages, kv * slab), "table": table,
          "row_start": torch.tensor(starts, dtype=torch.int32, device="cuda"),
          "kv_len": torch.tensor([length for length, _ in lengths], dtype=torch.int32, device="cuda")}
    rows = starts[-1]
    if case["op"] == "cache":
        st["k"] = (normal(rows, kv, dim) * torch.exp(normal(kv, dim, std=0.5))).to(dtype)
        st["v"] = normal(rows, kv, dim).to(dtype)
        # what is read back: the new tokens and up to 15 before them, so whatever a block's new scale changed
        held = [min(length, new + BLOCK - 1) for length, new in lengths]
        ends = [sum(held[:s]) for s in range(len(held) + 1)]
        st["held_start"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        st["k_out"] = torch.empty((ends[-1], kv, dim), dtype=dtype, device="cuda")
        st["v_out"] = torch.empty_like(st["k_out"])
        # which sequence and block each unit of the plain form is, and each row read back
        blocks = [(s, b) for s, (length, new) in enumerate(lengths)
                  for b in range((length - new) // BLOCK, (length - 1) // BLOCK + 1)]
        st["blocks"] = torch.tensor(blocks, dtype=torch.int64, device="cuda").T.contiguous()
        st["held"] = torch.repeat_interleave(torch.arange(len(held), device="cuda"),
                                             torch.tensor(held, device="cuda"), output_size=ends[-1])
        if own:
            from int8_quantized_matmul_gb300 import i2s
            cache = i2s.Kv8Cache(n_pages, kv, dim, page, data=st["pool"])
            new = i2s.Kv8Batch(st["row_start"], st["kv_len"], table, rows=rows, max_rows=max(news))
            back = i2s.Kv8Batch(st["held_start"], st["kv_len"], table, rows=ends[-1], max_rows=max(held))
            st["write"] = i2s.Kv8Write(cache, new, st["k"], st["v"])
            st["read"] = i2s.Kv8Read(cache, back, st["k_out"], st["v_out"])
        return st
    st["q"] = (normal(rows, case["q_heads"], dim) * 1.5).to(dtype)
    st["scale"] = dim ** -0.5
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty((rows, case["q_heads"]), device="cuda")
    st["row_seq"] = torch.repeat_interleave(torch.arange(len(news), device="cuda"),
                                            torch.tensor(news, device="cuda"), output_size=rows)
    if own:
        from int8_quantized_matmul_gb300 import i2s
        cache = i2s.Kv8Cache(n_pages, kv, dim, page, data=st["pool"])
        batch = i2s.Kv8Batch(st["row_start"], st["kv_len"], table, rows=rows, max_rows=max(news))
        st["call"] = i2s.Kv8Attention(cache, batch, st["q"], out=st["out"], scale=st["scale"], causal=True,
                                      window=case["window"], lse=st["lse"])
    return st


def run(st):
    if st["case"]["op"] == "rope":
        if own:
            st["call"]()
            return {"q": st["q_out"], "k": st["k_out"]}
        return _plain_rope(st)
    if st["case"]["op"] == "cache":
        if own:
            st["write"]()
            st["read"]()
            return {"k": st["k_out"], "v": st["v_out"]}
        return _plain_cache(st)
    if own:
        st["call"]()
        return {"out": st["out"], "lse": st["lse"]}
    return _plain_attend(st)


# -- the plain forms ------------------------------------------------------------------------------

def _plain_rope(st):
    case = st["case"]
    rot = case["rot"]
    # the angle in whole turns wraps at 64 bits; far positions need more than 32 of them
    turn = st["positions"].long()[:, None] * st["turns"][None, :]
    angle = turn.double() * (2 * math.pi / 2.0 ** 64)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(x, gamma):
        y = x.float()
        if gamma is not None:
            y = y * (1 / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6)) * gamma
        if case["pairs"] == "half":
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = y[..., :rot:2], y[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)

    return {"q": one(st["q"], st["gamma_q"]), "k": one(st["k"], st["gamma_k"])}


def _views(case, pool):
    """K codes, V codes [pages, heads, page, dim] and their scales [pages, heads, page / 16] in the pool."""
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    n, slab = pool.shape[0], _slab(dim, page)
    codes = pool.view(torch.int8).view(n, kv, slab)[:, :, :2 * page * dim].unflatten(2, (2, page, dim))
    scales = pool.view(torch.float32).view(n, kv, slab // 4)[:, :, page * dim // 2:page * dim // 2 + page // 8]
    scales = scales.unflatten(2, (2, page // BLOCK))
    return codes[:, :, 0], codes[:, :, 1], scales[:, :, 0], scales[:, :, 1]


def _plain_cache(st):
    case = st["case"]
    page = case["page"]
    kc, vc, ks, vs = _views(case, st["pool"])
    seq, block = st["blocks"]
    length, news = st["kv_len"].long(), (st["row_start"][1:] - st["row_start"][:-1]).long()
    start = (length - news)[seq][:, None]
    pos = block[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")
    fresh = (pos >= start) & (pos < length[seq][:, None])
    row = torch.where(fresh, pos - start + st["row_start"][seq].long()[:, None], 0)
    pg = st["table"].long()[seq, block * BLOCK // page]
    slot, sub = pos % page, block % (page // BLOCK)
    for x, codes, scales in ((st["k"], kc, ks), (st["v"], vc, vs)):
        value = torch.where(fresh[:, :, None, None], x[row].float(), 0.0)
        scale = value.abs().amax((1, 3)).clamp_min(1e-5)
        scale = scale / torch.full_like(scale, 127.0)  # by a tensor: a number's reciprocal would be multiplied
        before = scales[pg, :, sub]
        held = (start > block[:, None] * BLOCK)
        scale = torch.where(held, torch.maximum(scale, before), scale)
        was = codes[pg[:, None], :, slot]
        value = torch.where((pos < start)[:, :, None, None], was.float() * before[:, None, :, None], value)
        step = (value * (1.0 / scale)[:, None, :, None]).clamp(-127, 127).double()
        now = (step.sign() * (step.abs() + 0.5).floor()).to(torch.int8)
        same = (scale == before)[:, None, :, None] & ~fresh[:, :, None, None]
        codes[pg[:, None], :, slot] = torch.where((pos < length[seq][:, None])[:, :, None, None] & ~same, now, was)
        scales[pg, :, sub] = scale
    held = st["held"]
    n = st["held_start"].long()
    pos = length[held] - n[held + 1] + torch.arange(held.numel(), device="cuda")
    pg, slot = st["table"].long()[held, pos // page], pos % page
    return {name: (codes[pg, :, slot].float() * scales[pg, :, slot // BLOCK][:, :, None]).to(st["k"].dtype)
            for name, codes, scales in (("k", kc, ks), ("v", vc, vs))}


def _plain_attend(st):
    case = st["case"]
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    group, seqs, most = case["q_heads"] // kv, case["seqs"], case["new_hi"]
    kc, vc, ks, vs = _views(case, st["pool"])
    length = st["kv_len"].long()
    news = (st["row_start"][1:] - st["row_start"][:-1]).long()
    table = st["table"].long().clamp_min(0)
    keys = torch.arange(table.shape[1] * page, device="cuda")
    here = (keys < length[:, None])[:, None, :, None]

    def values(codes, scales):  # [seqs, kv, tokens, dim]
        x = codes[table].float() * scales[table].repeat_interleave(BLOCK, -1)[..., None]
        return torch.where(here, x.transpose(1, 2).reshape(seqs, kv, -1, dim), 0.0)

    row = torch.arange(st["q"].shape[0], device="cuda") - st["row_start"].long()[st["row_seq"]]
    q = torch.zeros((seqs, most, kv, group, dim), device="cuda")
    q[st["row_seq"], row] = st["q"].float().unflatten(1, (kv, group))
    q = q.permute(0, 2, 1, 3, 4).reshape(seqs, kv, most * group, dim)
    pos = (length - news)[:, None] + torch.arange(most, device="cuda")
    seen = (keys <= pos[:, :, None]) & here[:, :, :, 0]
    if case["window"]:
        seen &= keys > pos[:, :, None] - case["window"]
    seen = seen[:, None, :, None]
    score = (q @ values(kc, ks).transpose(2, 3)).unflatten(2, (most, group)) * st["scale"]
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-1e30)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = ((score.flatten(2, 3) @ values(vc, vs)).unflatten(2, (most, group)) / total)
    lse = (top + total.log())[..., 0]
    at = (st["row_seq"], slice(None), row)
    return {"out": out[at].flatten(1, 2).to(st["q"].dtype), "lse": lse[at].flatten(1, 2)}


# -- the definitions in 64 bits --------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        rot, far = case["rot"], st["positions"].tolist()
        turns = [t % (1 << 64) for t in st["turns"].tolist()]
        angle = torch.tensor([[(p * t % (1 << 64)) / 2.0 ** 64 for t in turns] for p in far], dtype=torch.float64,
                             device="cuda") * 2 * math.pi
        unit = torch.polar(torch.ones_like(angle), angle)[:, None]
        got = {}
        for name in ("q", "k"):
            y = st[name].double()
            gamma = st["gamma_" + name]
            if gamma is not None:
                y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * gamma.double()
            if case["pairs"] == "half":
                z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * unit
                turned = torch.cat([z.real, z.imag], -1)
            else:
                turned = torch.view_as_real(torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous())
                                            * unit).flatten(-2)
            got[name] = torch.cat([turned, y[..., rot:]], -1)
        return got
    kv, dim, page, slab = case["kv_heads"], case["dim"], case["page"], _slab(case["dim"], case["page"])
    pool = st["pool"].view(-1, kv, slab)
    plane = page * dim

    def cached(s, last, which):
        """Codes [tokens, kv, dim] and scales [tokens, kv] of positions 0 .. last - 1 of sequence s."""
        used = pool[st["table"][s, :-(-last // page)].long()]
        codes = used[:, :, which * plane:(which + 1) * plane].contiguous().view(torch.int8)
        codes = codes.view(-1, kv, page, dim).transpose(1, 2).reshape(-1, kv, dim)[:last]
        at = 2 * plane + which * page // 4
        scales = used[:, :, at:at + page // 4].contiguous().view(torch.float32)
        scales = scales.transpose(1, 2).reshape(-1, kv)
        return codes, scales.repeat_interleave(BLOCK, 0)[:last]

    lengths, row = _lengths(case), 0
    if case["op"] == "cache":
        got = {"k": [], "v": []}
        for s, (length, new) in enumerate(lengths):
            for which, name in enumerate(("k", "v")):
                codes, scales = cached(s, length, which)
                start, codes = length - new, codes.double()
                values = codes * scales.double()[:, :, None]
                values[start:] = st[name][row:row + new].double()
                lo = start // BLOCK * BLOCK
                some = torch.nn.functional.pad(values[lo:], (0, 0, 0, 0, 0, -length % BLOCK)).unflatten(0, (-1, BLOCK))
                new_some = some.clone()
                new_some[0, :start - lo] = 0
                # the stored numbers are binary32: each step below is rounded to it as the definition says
                scale = (new_some.abs().amax((1, 3)).clamp_min(float(torch.tensor(1e-5))) / 127).float()
                if start > lo:
                    scale[0] = torch.maximum(scale[0], scales[lo])
                    some[0, :start - lo] = some[0, :start - lo].float().double()
                inv = (1 / scale.double()).float().double()
                q = (some * inv[:, None, :, None]).float().double().clamp(-127, 127)
                q = q.sign() * (q.abs() + 0.5).floor()
                back = (q * scale.double()[:, None, :, None]).flatten(0, 1)[:length - lo]
                if start > lo:
                    keep = (scale[0] == scales[lo])[None, :, None]
                    back[:start - lo] = torch.where(keep, values[lo:start], back[:start - lo])
                values[lo:] = back
                got[name].append(values[length - min(length, new + BLOCK - 1):])
            row += new
        return {name: torch.cat(parts) for name, parts in got.items()}
    group = case["q_heads"] // kv
    out, lse = [], []
    for s, (length, new) in enumerate(lengths):
        q = st["q"][row:row + new].double().unflatten(1, (kv, group))
        row += new
        (kc, ks), (vc, vs) = cached(s, length, 0), cached(s, length, 1)
        pos = torch.arange(length - new, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")
        hidden = key > pos
        if case["window"]:
            hidden |= key <= pos - case["window"]
        heads = []
        for h in range(kv):
            k = kc[:, h].double() * ks[:, h, None].double()
            v = vc[:, h].double() * vs[:, h, None].double()
            for g in range(group):
                score = (q[:, h, g] @ k.T * st["scale"]).masked_fill_(hidden, -math.inf)
                total = torch.logsumexp(score, -1)
                heads.append((torch.softmax(score, -1) @ v, total))
        out.append(torch.stack([o for o, _ in heads], 1))
        lse.append(torch.stack([t for _, t in heads], 1))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
