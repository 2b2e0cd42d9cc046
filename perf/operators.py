"""The serving operators that stand beside the GEMV, as measured cases.

Four operators, each reached through the package's public entry points:

``linear``     rows of x rounded to 8-bit integers (a scale per token), then the
               product with 8-bit weights (a scale per output channel): the
               linear layer for more tokens than the GEMV takes.
``append``     new K and V rows rounded to 4 bits into the pages of a cache.
``attention``  softmax attention of each sequence's newest tokens over its
               4-bit cache; optionally adds every token's attention weight to a
               running mass.
``evict``      keeps the newest tokens and those of the largest mass, copied to
               fresh pages in their order.

The cache is held in pages. A page of ``page`` tokens is, for each KV head and
for K then V, one block of ``page * (dim / 2 + 4 * dim / group)`` bytes: the
4-bit codes of its tokens, then (scale, lowest value) of each token's groups.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}


def _lin(name, n, inp, out, x, y):
    return {"name": name, "op": "linear", "n": n, "in": inp, "out": out, "x": x, "y": y}


def _cache(q_heads, heads, dim, page, group, dtype):
    return {"q_heads": q_heads, "heads": heads, "dim": dim, "page": page, "group": group, "dtype": dtype}


def listed():
    return [
        # q_proj of one decoded token: the smallest call, latency and one pass over the weights
        _lin("linear_1x4096x4096", 1, 4096, 4096, "fp16", "fp16"),
        # gate and up stacked, for a decode batch of 24 sequences: bound by the weights' bytes
        _lin("linear_24x4096x28672", 24, 4096, 28672, "fp16", "fp16"),
        # a ragged prompt chunk on sizes that no tile divides, fp32 result
        _lin("linear_333x5003x1285_bf16", 333, 5003, 1285, "bf16", "fp32"),
        # down_proj of a 4096-token prompt: bound by the tensor cores
        _lin("linear_4096x14336x4096", 4096, 14336, 4096, "fp16", "fp16"),
        # one decoded token's K and V into the cache: latency
        {"name": "append_1", "op": "append", "batch": 1, "new": 1, "len": 1000, **_cache(32, 8, 128, 64, 128, "fp16")},
        # the prompts of 4 sequences, starting inside a page
        {"name": "append_4x4099_bf16", "op": "append", "batch": 4, "new": 4099, "len": 37, **_cache(40, 10, 128, 32, 32, "bf16")},
        # one sequence's decode step at a short context: latency
        {"name": "attention_1x777", "op": "attention", "batch": 1, "new": 1, "len": 777, "mass": False, **_cache(32, 8, 128, 16, 128, "fp16")},
        # a decode batch with ragged contexts, one of them empty
        {"name": "attention_16x8192", "op": "attention", "batch": 16, "new": 1, "len": 8192, "mass": False, **_cache(32, 8, 128, 64, 128, "fp16")},
        # two long contexts: bound by the cache's bytes
        {"name": "attention_2x120001_bf16", "op": "attention", "batch": 2, "new": 1, "len": 120001, "mass": False, **_cache(40, 10, 128, 64, 64, "bf16")},
        # four tokens checked at once, one KV head for each query head, with the mass that eviction needs
        {"name": "attention_8x4001_new4_mass", "op": "attention", "batch": 8, "new": 4, "len": 4001, "mass": True, **_cache(32, 32, 128, 32, 128, "fp16")},
        # a short cache halved
        {"name": "evict_1x1000", "op": "evict", "batch": 1, "len": 1000, "budget": 500, "recent": 63, **_cache(32, 8, 128, 16, 128, "fp16")},
        # a batch of long caches cut to a fixed budget
        {"name": "evict_8x32768", "op": "evict", "batch": 8, "len": 32768, "budget": 2048, "recent": 256, **_cache(32, 8, 128, 64, 64, "bf16")},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "append", "attention", "attention", "evict"])
    if op == "linear":
        n, inp, out = _log(rng, 1, 8192), _log(rng, 40, 17920), _log(rng, 64, 28672)
        if n * inp * out > 2.4e11:
            n = max(1, int(2.4e11 / (inp * out)))
        return {"op": op, "n": n, "in": inp, "out": out, "x": rng.choice(["fp16", "bf16"]), "y": rng.choice(["fp16", "bf16", "fp32"])}
    dim = rng.choice([64, 128, 128])
    heads = rng.choice([1, 2, 5, 8, 8, 10, 32])
    per = rng.choice([1, 2, 4, 4, 5, 7, 8])
    case = _cache(heads * per, heads, dim, rng.choice([16, 32, 64, 128]), rng.choice([g for g in (32, 64, 128) if g <= dim]), rng.choice(["fp16", "bf16"]))
    batch = _log(rng, 1, 32)
    if op == "append":
        new = max(1, min(_log(rng, 1, 8192), 160000 // (batch * heads)))
        return {"op": op, "batch": batch, "new": new, "len": rng.randrange(0, 500), **case}
    length = max(1, min(_log(rng, 1, 131072), 2400000 // (batch * heads)))
    if op == "attention":
        return {"op": op, "batch": batch, "new": rng.choice([1, 1, 2, 3, 5, 8]), "len": length, "mass": rng.random() < 0.4, **case}
    budget = min(max(1, length - rng.randrange(0, length)), 140000 // (batch * heads))
    return {"op": op, "batch": batch, "len": length, "budget": budget, "recent": rng.randrange(0, budget + 1), **case}


# ------------------------------------------------------------------ inputs

def _lens(case):
    """Cached tokens of each sequence, the newest ones included: the first has
    them all, the others fewer; of four or more sequences the third is empty."""
    b, n = case["batch"], case["len"]
    lens = [n - (i * 7 * n) // (b * 8) for i in range(b)]
    if b >= 4 and case["op"] == "attention":
        lens[2] = 0
    return lens


def _pages_of(case):
    """Pages that the longest sequence fills."""
    tokens = case["len"] + (case["new"] if case["op"] == "append" else 0)
    return -(-tokens // case["page"])


def _gen(seed, what):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 16 + what)


def _normal(seed, what, shape, dtype):
    return torch.randn(shape, generator=_gen(seed, what), device=DEV, dtype=torch.float32).to(dtype)


def _kv(case, seed, tokens):
    """K and V [batch, tokens, heads, dim]: a few of K's channels are much
    larger than the others, and every channel of it has an offset."""
    shape = (case["batch"], tokens, case["heads"], case["dim"])
    g = _gen(seed, 1)
    size = 0.5 + torch.rand((1, 1) + shape[2:], generator=g, device=DEV)
    size = torch.where(torch.rand(size.shape, generator=g, device=DEV) < 0.04, size * 5, size)
    mean = torch.randn(size.shape, generator=g, device=DEV) * 0.7
    k = torch.randn(shape, generator=g, device=DEV).mul_(size).add_(mean).to(DT[case["dtype"]])
    return k, _normal(seed, 2, shape, DT[case["dtype"]])


def _mass(case, seed):
    """Accumulated weights [batch, heads, tokens]: heavy-tailed, with ties."""
    m = torch.randn((case["batch"], case["heads"], _pages_of(case) * case["page"]), generator=_gen(seed, 3), device=DEV)
    return torch.floor(torch.exp(m * 2) * 64) / 64


def _scores(n, seed, what):
    return torch.rand(n, generator=_gen(seed, what), device=DEV)


def prepare(case, seed):
    s = dict(case)
    if case["op"] == "linear":
        n, inp, out = case["n"], case["in"], case["out"]
        s["x"] = _normal(seed, 0, (n, inp), DT[case["x"]])
        w = _normal(seed, 4, (out, inp), torch.float32) * 0.02
        s["ws"] = w.abs().amax(1) / 127
        row = -(-inp // 128) * 128  # rows of 8-bit values are padded with zeros to 128 bytes
        s["wq"] = torch.zeros((out, row), dtype=torch.int8, device=DEV)
        s["wq"][:, :inp] = torch.round(w / s["ws"][:, None]).to(torch.int8)
        s["xq"] = torch.empty((n, row), dtype=torch.int8, device=DEV)
        s["xs"] = torch.empty(n, dtype=torch.float32, device=DEV)
        s["out"] = torch.empty((n, out), dtype=DT[case["y"]], device=DEV)
        return s
    batch, heads, dim, page, group = (case[k] for k in ("batch", "heads", "dim", "page", "group"))
    dtype, ng = DT[case["dtype"]], dim // group
    per = _pages_of(case)
    fresh = -(-case["budget"] // page) if case["op"] == "evict" else 0
    total = batch * (per + fresh)
    order = torch.argsort(_scores(total, seed, 5)).to(torch.int32)
    s["table"] = order[: batch * per].reshape(batch, per).contiguous()
    s["pages"] = torch.zeros((total, heads, 2, page * (dim // 2 + 4 * ng)), dtype=torch.uint8, device=DEV)
    s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
    if case["op"] == "append":
        k, v = _kv(case, seed, case["new"])
        s["k"], s["v"] = k.reshape(-1, heads * dim), v.reshape(-1, heads * dim)
        s["lens"] = s["lens"] + case["new"]  # as attention takes them: the new tokens included
        s["starts"] = s["lens"] - case["new"]
        s["k_out"], s["v_out"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        return s
    k, v = _kv(case, seed, per * page)
    _write(s, k, v, torch.zeros(batch, dtype=torch.int32, device=DEV))
    if case["op"] == "attention":
        s["q"] = _normal(seed, 6, (batch * case["new"], case["q_heads"] * dim), dtype)
        s["out"] = torch.empty_like(s["q"])
        if case["mass"]:
            s["mass0"] = _mass(case, seed)
            s["mass"] = s["mass0"].clone()
        return s
    s["dst_table"] = order[batch * per:].reshape(batch, fresh).contiguous()
    s["mass"] = _mass(case, seed)
    s["kept"] = torch.empty((batch, heads, case["budget"]), dtype=torch.int32, device=DEV)
    s["new_lens"] = torch.empty(batch, dtype=torch.int32, device=DEV)
    s["new_mass"] = torch.empty((batch, heads, fresh * page), dtype=torch.float32, device=DEV)
    s["k_out"] = torch.empty((batch * case["budget"], heads * dim), dtype=dtype, device=DEV)
    s["v_out"] = torch.empty_like(s["k_out"])
    return s


# ------------------------------------------------------------- plain forms

def _rounded4(x, group):
    """Codes, scale and lowest value of x [..., dim] in groups along dim."""
    g = x.unflatten(-1, (-1, group))
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((hi.double() - lo.double()) / 15).to(x.dtype)
    # 64 bits: (x - lo) / s decides a rounding, and x - lo alone can need more than 32
    u = torch.round((g.double() - lo.double()[..., None]) / s.double()[..., None]).clamp(0, 15)
    u = torch.where(s[..., None] == 0, torch.zeros((), dtype=u.dtype, device=u.device), u)
    return u.flatten(-2).to(torch.uint8), s, lo


def _parts(s):
    """Views of the pages: codes and (scale, lowest) of K and V, each [page, head, token, ...]."""
    dim, page, ng = s["dim"], s["page"], s["dim"] // s["group"]
    codes = s["pages"][..., : page * dim // 2].unflatten(-1, (page, dim // 2))
    meta = s["pages"][..., page * dim // 2:].view(DT[s["dtype"]]).unflatten(-1, (page, ng, 2))
    return codes, meta


def _put(s, codes, meta, x, which, pid, slot):
    u, scale, lo = _rounded4(x, s["group"])
    blocks = (-1, 4, 8) if which == 0 else (-1, 8, 4)
    # a row's codes: 32 channels after 32, those of one reading lane together
    u = u.unflatten(-1, blocks).transpose(-3, -2).flatten(-3)
    codes[pid, :, which, slot] = u[..., 0::2] | (u[..., 1::2] << 4)
    meta[pid, :, which, slot] = torch.stack([scale, lo], -1)


def _write(s, k, v, starts):
    """k, v [batch, new, heads, dim] into the pages, from each sequence's start on."""
    pos = starts.long()[:, None] + torch.arange(k.shape[1], device=k.device)
    pid, slot = torch.gather(s["table"].long(), 1, pos // s["page"]), pos % s["page"]
    codes, meta = _parts(s)
    _put(s, codes, meta, k, 0, pid, slot)
    _put(s, codes, meta, v, 1, pid, slot)


def _values(s, which, table, first, count):
    """fp32 values [batch, count, heads, dim] of positions first .. first + count - 1."""
    pos = first.long()[:, None] + torch.arange(count, device=table.device)
    pid, slot = torch.gather(table.long(), 1, pos // s["page"]), pos % s["page"]
    codes, meta = _parts(s)
    b, m = codes[pid, :, which, slot], meta[pid, :, which, slot].float()
    u = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    blocks = (4, -1, 8) if which == 0 else (8, -1, 4)
    u = u.unflatten(-1, blocks).transpose(-3, -2).flatten(-3)
    u = u.unflatten(-1, (-1, s["group"])).float()
    return (m[..., 1][..., None] + m[..., 0][..., None] * u).flatten(-2)


def _linear(s):
    x = s["x"]
    a = x.abs().amax(1, keepdim=True)
    # 64 bits: the quotient decides a rounding
    q = torch.round(x.double() * 127 / a.double()).float()
    q = torch.where(a == 0, torch.zeros((), device=q.device), q)
    y = q @ s["wq"][:, : s["in"]].float().t()
    s["out"].copy_(y * (a.float() / 127) * s["ws"])
    return s["out"]


def _append(s):
    shape = (s["batch"], s["new"], s["heads"], s["dim"])
    _write(s, s["k"].view(shape), s["v"].view(shape), s["starts"])
    s["k_out"].copy_(_values(s, 0, s["table"], s["starts"], s["new"]).view_as(s["k_out"]))
    s["v_out"].copy_(_values(s, 1, s["table"], s["starts"], s["new"]).view_as(s["v_out"]))
    return s["k_out"], s["v_out"]


def _attention(s):
    b, n, hk, dim = s["batch"], s["new"], s["heads"], s["dim"]
    zero = torch.zeros_like(s["lens"])
    k, v = (_values(s, i, s["table"], zero, s["len"]).transpose(1, 2) for i in (0, 1))  # [b, hk, t, dim]
    q = s["q"].float().view(b, n, hk, -1, dim).permute(0, 2, 1, 3, 4)  # [b, hk, n, per, dim]
    per = q.shape[3]
    sc = (q.reshape(b, hk, n * per, dim) @ k.transpose(2, 3)).view(b, hk, n, per, -1) / math.sqrt(dim)
    limit = s["lens"][:, None] - (n - 1) + torch.arange(n, device=q.device)  # [b, n]
    seen = torch.arange(s["len"], device=q.device) < limit[..., None]  # [b, n, t]
    seen = seen[:, None, :, None, :]
    sc = sc.masked_fill(~seen, -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = p.view(b, hk, n * per, -1) @ v
    s["out"].copy_(o.view(b, hk, n, per, dim).permute(0, 2, 1, 3, 4).reshape(b * n, -1))
    if s["mass"] is not False:
        s["mass"].copy_(s["mass0"])
        s["mass"][..., : s["len"]] += p.sum((2, 3))
        return s["out"], s["mass"]
    return s["out"]


def _evict(s):
    b, h, budget, page = s["batch"], s["heads"], s["budget"], s["page"]
    cap = s["mass"].shape[2]
    pos, lens = torch.arange(cap, device=s["mass"].device), s["lens"][:, None, None]
    key = torch.where(pos >= lens - s["recent"], math.inf, s["mass"])
    key = torch.where(pos >= lens, -math.inf, key)
    keep = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :budget]
    keep = torch.sort(torch.where(keep < lens, keep, cap), dim=-1)[0]  # in their order, the missing ones last
    new_lens = s["lens"].clamp_max(budget)
    there = keep < cap
    at = torch.where(there, keep, 0)
    seq, head = torch.arange(b, device=at.device)[:, None, None], torch.arange(h, device=at.device)[:, None]
    src, dst = s["table"].long()[seq, at // page], torch.arange(budget, device=at.device)
    to = s["dst_table"].long()[seq, dst // page].expand_as(at)
    codes, meta = _parts(s)
    slot, head = (dst % page).expand_as(at), head.expand_as(at)
    where = (to[there], head[there], slot[there])
    frm = (src[there], head[there], (at % page)[there])
    codes[where[0], where[1], :, where[2]] = codes[frm[0], frm[1], :, frm[2]]
    meta[where[0], where[1], :, where[2]] = meta[frm[0], frm[1], :, frm[2]]
    s["kept"].copy_(torch.where(there, keep, -1))
    s["new_lens"].copy_(new_lens)
    s["new_mass"].zero_()
    s["new_mass"][..., :budget] = torch.where(there, torch.gather(s["mass"], 2, at), 0.0)
    zero, inside = torch.zeros_like(new_lens), (dst < new_lens[:, None])[..., None, None]
    for_k, for_v = (torch.where(inside, _values(s, i, s["dst_table"], zero, budget), 0.0) for i in (0, 1))
    s["k_out"].copy_(for_k.view_as(s["k_out"]))
    s["v_out"].copy_(for_v.view_as(s["v_out"]))
    return s["kept"], s["new_lens"], s["new_mass"], s["k_out"], s["v_out"]


# ------------------------------------------------------------ the entry points

def _run_own(s):
    import quantized_gemv_stagq_b200 as Q

    if s["op"] == "linear":
        Q.stagq_quantize_i8(s["x"], s["xq"], s["xs"])
        Q.stagq_gemm_i8(s["xq"], s["xs"], s["wq"], s["ws"], s["in"], s["out"])
        return s["out"]
    cache = Q.KVCache(s["pages"], s["heads"], s["dim"], s["page"], s["group"], DT[s["dtype"]])
    if s["op"] == "append":
        Q.stagq_kv_append(cache, s["k"], s["v"], s["table"], s["starts"], s["new"])
        Q.stagq_kv_read(cache, s["table"], s["lens"], s["k_out"], s["v_out"], s["new"], starts=s["starts"])
        return s["k_out"], s["v_out"]
    if s["op"] == "attention":
        if s["mass"] is False:
            Q.stagq_kv_attention(cache, s["q"], s["table"], s["lens"], s["out"], n_new=s["new"])
            return s["out"]
        s["mass"].copy_(s["mass0"])
        Q.stagq_kv_attention(cache, s["q"], s["table"], s["lens"], s["out"], n_new=s["new"], mass=s["mass"])
        return s["out"], s["mass"]
    Q.stagq_kv_evict(cache, s["table"], s["lens"], s["mass"], s["dst_table"], s["budget"], s["recent"],
                     s["kept"], s["new_lens"], s["new_mass"])
    Q.stagq_kv_read(cache, s["dst_table"], s["new_lens"], s["k_out"], s["v_out"], s["budget"])
    return s["kept"], s["new_lens"], s["new_mass"], s["k_out"], s["v_out"]


def run(state):
    if own:
        return _run_own(state)
    return {"linear": _linear, "append": _append, "attention": _attention, "evict": _evict}[state["op"]](state)


# ------------------------------------------------------------------ work, exact

def work(case):
    if case["op"] == "linear":
        n, inp, out = case["n"], case["in"], case["out"]
        return {"bytes": n * inp * SIZE[case["x"]] + out * inp + 4 * out + n * out * SIZE[case["y"]], "flops": 2 * n * inp * out}
    heads, dim = case["heads"], case["dim"]
    row = 2 * heads * (dim // 2 + 4 * (dim // case["group"]))  # a cached token's bytes, K and V
    raw = 2 * heads * dim * 2  # the same as fp16 or bf16
    if case["op"] == "append":
        n = case["batch"] * case["new"]
        return {"bytes": n * (raw + row + raw), "flops": 8 * n * heads * dim}  # the last: the values are returned
    tokens = sum(_lens(case))
    if case["op"] == "attention":
        q = 2 * case["batch"] * case["new"] * case["q_heads"] * dim * 2
        flops = 4 * tokens * case["new"] * case["q_heads"] * dim
        return {"bytes": tokens * row + q + (8 * tokens * heads if case["mass"] else 0), "flops": flops}
    kept = sum(min(n, case["budget"]) for n in _lens(case))
    return {"bytes": 4 * tokens * heads + kept * (2 * row + 12 * heads + raw), "flops": 4 * tokens * heads}


def _exact4(x, group):
    """The values that x [..., dim] stands for after rounding to 4 bits, in 64 bits."""
    g = x.double().reshape(*x.shape[:-1], x.shape[-1] // group, group)
    lo = g.min(-1, keepdim=True)[0]
    s = ((g.max(-1, keepdim=True)[0] - lo) / 15).to(x.dtype).double()
    u = torch.where(s > 0, ((g - lo) / s).round().clamp(0, 15), 0.0)
    return (lo + s * u).reshape(x.shape)


def exact(case, seed):
    if case["op"] == "linear":
        x = _normal(seed, 0, (case["n"], case["in"]), DT[case["x"]]).double()
        w = _normal(seed, 4, (case["out"], case["in"]), torch.float32) * 0.02
        ws = w.abs().amax(1) / 127
        wq = torch.round(w / ws[:, None]).double()
        a = x.abs().max(1, keepdim=True)[0]
        q = torch.where(a > 0, (127 * x / a).round(), 0.0)
        return (q @ wq.t()) * (a / 127) * ws.double()
    batch, heads, dim, group = case["batch"], case["heads"], case["dim"], case["group"]
    if case["op"] == "append":
        k, v = _kv(case, seed, case["new"])
        return tuple(_exact4(x, group).reshape(-1, heads * dim) for x in (k, v))
    k, v = _kv(case, seed, _pages_of(case) * case["page"])
    lens = _lens(case)
    if case["op"] == "attention":
        n, per = case["new"], case["q_heads"] // heads
        q = _normal(seed, 6, (batch * n, case["q_heads"] * dim), DT[case["dtype"]]).double().reshape(batch, n, heads, per, dim)
        out = torch.zeros_like(q)
        mass = _mass(case, seed).double() if case["mass"] else None
        for b in range(batch):
            for h in range(heads):
                kk, vv = (_exact4(x[b, : lens[b], h], group) for x in (k, v))
                for j in range(n):
                    m = lens[b] - (n - 1 - j)
                    if m > 0:
                        p = torch.softmax(q[b, j, h] @ kk[:m].t() * dim ** -0.5, -1)
                        out[b, j, h] = p @ vv[:m]
                        if mass is not None:
                            mass[b, h, :m] += p.sum(0)
        out = out.reshape(batch * n, -1)
        return out if mass is None else (out, mass)
    mass, budget = _mass(case, seed), case["budget"]
    kept = torch.full((batch, heads, budget), -1, dtype=torch.int32, device=DEV)
    fresh = -(-budget // case["page"]) * case["page"]
    new_mass = torch.zeros((batch, heads, fresh), dtype=torch.float64, device=DEV)
    out = [torch.zeros((batch, budget, heads, dim), dtype=torch.float64, device=DEV) for _ in (k, v)]
    for b in range(batch):
        old = max(0, lens[b] - case["recent"])
        for h in range(heads):
            idx = torch.arange(lens[b], device=DEV)
            if lens[b] > budget:
                # value first, then the lower index: one key that has no ties
                m = mass[b, h, :old].double()
                rank = torch.argsort(torch.argsort(-m, stable=True))
                idx = torch.cat([idx[:old][rank < budget - case["recent"]], idx[old:]])
            kept[b, h, : len(idx)] = idx.to(torch.int32)
            new_mass[b, h, : len(idx)] = mass[b, h, idx].double()
            for o, x in zip(out, (k, v)):
                o[b, : len(idx), h] = _exact4(x[b, idx, h], group)
    new_lens = torch.tensor([min(x, budget) for x in lens], dtype=torch.int32, device=DEV)
    return kept, new_lens, new_mass, out[0].reshape(-1, heads * dim), out[1].reshape(-1, heads * dim)
