"""Measured cases of the operators between a decoder layer's projections.

Four operators, as a decoder with a paged key-value cache calls them in every
step: ``assign`` turns request lengths into block tables, slots and positions;
``append`` rotates the new tokens' queries and keys and writes keys and values
into their slots; ``attention`` attends with one new token per request over
the paged cache; ``norm`` adds a block's output to the residual stream (its
norm, gate and scale before, the next block's norm behind).

``run`` computes them with elementary torch operations, or, where ``own`` is
true, through ``ternary_weight_decoder_b200.api``.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    # The decoder of the projection sweeps: 12 query heads over 2 KV heads of
    # 128, hidden size 1536.
    qwen = dict(heads=12, kv_heads=2, head_dim=128)
    return [
        # One step of 32 running requests: each takes one more token.
        dict(name="assign_step_32", op="assign", requests=32, page=16, max_len=4096,
             rows=32, mix="step"),
        # A scheduler's turn in a full server: prompts come in, finished
        # requests hand their pages back, the others take one token.
        dict(name="assign_turn_1024", op="assign", requests=1024, page=16, max_len=4096,
             rows=65536, mix="turn"),
        # The new tokens of one step of 32 requests, four rows of them padding.
        dict(name="append_step_32", op="append", rows=32, pad=4, dtype="bf16", page=16,
             rotary=128, interleaved=False, far=32768, **qwen),
        # A chunk of prompts, far into long contexts.
        dict(name="append_prompt_8192", op="append", rows=8192, pad=0, dtype="f16", page=64,
             rotary=128, interleaved=False, far=1048576, **qwen),
        # The same into a cache of 8-bit codes, with half of each head rotated.
        dict(name="append_codes_1000", op="append", rows=1000, pad=24, dtype="i8", page=32,
             rotary=64, interleaved=True, far=131072, **qwen),
        # A short utterance: one request, a few hundred frames.
        dict(name="attend_short_1", op="attention", requests=1, min_len=300, max_len=300,
             page=16, dtype="bf16", window=0, empty=0, **qwen),
        # One request over a very long context: all of the GPU on two heads.
        dict(name="attend_long_1", op="attention", requests=1, min_len=131072, max_len=131072,
             page=64, dtype="bf16", window=0, empty=0, **qwen),
        # A step of 33 requests of very different lengths, one not begun yet.
        dict(name="attend_step_33", op="attention", requests=33, min_len=1, max_len=4096,
             page=16, dtype="f16", window=0, empty=1, **qwen),
        # A full server on a cache of 8-bit codes.
        dict(name="attend_codes_256", op="attention", requests=256, min_len=512, max_len=16384,
             page=64, dtype="i8", window=0, empty=0, **qwen),
        # One token between two blocks.
        dict(name="norm_token_1", op="norm", rows=1, width=1536, post="", pre="rms", gate="",
             alpha=1.0, codes=False),
        # A prompt between two blocks with a norm on both sides and a gate.
        dict(name="norm_prompt_4096", op="norm", rows=4096, width=1536, post="rms", pre="rms",
             gate="channel", alpha=0.5, codes=False),
        # Wide rows with mean and bias, gated by token, quantised for the next projection.
        dict(name="norm_codes_1000", op="norm", rows=1000, width=8960, post="layer", pre="layer",
             gate="token", alpha=1.0, codes=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((12, 2, 128), (2, 1, 128), (2, 2, 128), (14, 2, 64), (8, 8, 64), (16, 2, 96), (9, 3, 80),
         (8, 1, 256), (5, 5, 128), (16, 1, 128), (32, 4, 128))


def draw(rng):
    op = rng.choice(("assign", "append", "attention", "norm"))
    heads, kv_heads, head_dim = rng.choice(HEADS)
    shape = dict(heads=heads, kv_heads=kv_heads, head_dim=head_dim)
    page = rng.choice((8, 16, 32, 48, 64, 128, 256))
    if op == "assign":
        requests, mix = _log(rng, 1, 2048), rng.choice(("step", "turn"))
        max_len = _log(rng, 64, 4096)
        rows = requests + rng.randrange(8) if mix == "step" else \
            requests * max(2, min(max_len, 65536 // requests) // 2) + rng.randrange(64)
        return dict(op=op, requests=requests, page=page, max_len=max_len, rows=rows, mix=mix)
    if op == "append":
        rows = _log(rng, 2, 6000)
        return dict(op=op, rows=rows, pad=rng.randrange(1 + min(rows - 1, 30)),
                    dtype=rng.choice(("bf16", "f16", "i8")), page=page,
                    rotary=rng.choice((head_dim, head_dim // 16 * 8, 0)),
                    interleaved=rng.random() < 0.5, far=_log(rng, 16, 1048576), **shape)
    if op == "attention":
        requests = _log(rng, 1, 256)
        most = min(131072, 2 ** 27 // (requests * kv_heads * head_dim))
        max_len = _log(rng, 2, most)
        return dict(op=op, requests=requests, min_len=_log(rng, 1, max_len), max_len=max_len,
                    page=page, dtype=rng.choice(("bf16", "f16", "i8")),
                    window=rng.choice((0, 0, _log(rng, 1, max_len))),
                    empty=rng.randrange(1 + requests // 4), **shape)
    rows = _log(rng, 1, 4096)
    return dict(op=op, rows=rows, width=min(_log(rng, 64, 16384), 6000000 // rows),
                post=rng.choice(("", "rms", "layer")), pre=rng.choice(("rms", "layer")),
                gate=rng.choice(("", "channel", "token")), alpha=rng.choice((1.0, 0.5, 0.125)),
                codes=rng.random() < 0.25)


# ------------------------------------------------------------------ inputs
def _generator(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _lengths(case):
    """The case's lengths, spread over the logarithm of its range."""
    n, lo, hi = case["requests"], case["min_len"], case["max_len"]
    got = [round(lo * (hi / lo) ** ((i + 0.5) / n)) for i in range(n)]
    return [0] * case["empty"] + got[case["empty"]:]


def _pools(case, pages, g):
    """Key and value pools [pages, page, kv_heads, head_dim], and the codes' scales."""
    size = (pages, case["page"], case["kv_heads"], case["head_dim"])
    out = {}
    for name in ("k", "v"):
        if case["dtype"] == "i8":
            codes = torch.randn(size, device="cuda", generator=g, dtype=torch.float16)
            out[name] = codes.mul_(40).round_().clamp_(-127, 127).to(torch.int8)
            out[name + "_scale"] = torch.rand(size[:3], device="cuda", generator=g) * 0.02 + 0.015
        else:
            out[name] = torch.randn(size, device="cuda", generator=g, dtype=DTYPES[case["dtype"]])
            out[name + "_scale"] = None
    return out


def prepare(case, seed):
    g, c = _generator(seed, "cuda"), _generator(seed, "cpu")
    s = {"case": dict(case)}
    if case["op"] == "assign":
        n, page, top = case["requests"], case["page"], case["max_len"]
        width = -(-top // page)
        old = torch.randint(0, top // 2 + 1, (n,), generator=c)
        if case["mix"] == "step":
            delta = torch.ones(n, dtype=torch.int64)
        else:
            delta = torch.ones(n, dtype=torch.int64)
            kind = torch.rand(n, generator=c)
            long = max(1, min(top // 2, case["rows"] // n))
            fresh = torch.randint(1, long + 1, (n,), generator=c)
            delta = torch.where(kind < 0.5, fresh, delta)
            delta = torch.where(kind > 0.8, -old, delta)
        held = (old + page - 1) // page
        pages = torch.randperm(n * width, generator=c)
        table = torch.full((n, width), -1, dtype=torch.int64)
        mine = torch.arange(width)[None, :] < held[:, None]
        used = int(held.sum())
        table[mine] = pages[:used]
        free = torch.full((n * width,), -1, dtype=torch.int64)
        free[:n * width - used] = pages[used:]
        for name, t in (("lengths", old), ("delta", delta), ("block_table", table),
                        ("free_pages", free), ("free_count", torch.tensor([n * width - used]))):
            s[name] = t.to(torch.int32).cuda()
        return s
    if case["op"] == "append":
        n, d, page = case["rows"], case["head_dim"], case["page"]
        real = n - case["pad"]
        pages = -(-real // page) + 1
        s.update(_pools(case, pages, g))
        # queries, keys and values as slices of the projections' one buffer
        qkv = torch.randn((n, (case["heads"] + 2 * case["kv_heads"]) * d), device="cuda", generator=g)
        s["q"], s["k_new"], s["v_new"] = qkv.split(
            [case["heads"] * d, case["kv_heads"] * d, case["kv_heads"] * d], dim=1)
        slots = torch.full((n,), -1, dtype=torch.int64)
        slots[:real] = torch.randperm(pages * page, generator=c)[:real]
        positions = torch.randint(0, case["far"], (n,), generator=c)
        positions[real:] = 0
        s["slots"], s["positions"] = (t.to(torch.int32).cuda() for t in (slots, positions))
        half = torch.arange(case["rotary"] // 2, dtype=torch.float64)
        s["inv_freq"] = (1e6 ** (-2 * half / max(1, case["rotary"]))).cuda()
        return s
    if case["op"] == "attention":
        lengths = torch.tensor(_lengths(case))[torch.randperm(case["requests"], generator=c)]
        page = case["page"]
        held = (lengths + page - 1) // page
        width, used = -(-case["max_len"] // page), int(held.sum())
        s.update(_pools(case, used + 1, g))
        table = torch.zeros((case["requests"], width), dtype=torch.int64)
        table[torch.arange(width)[None, :] < held[:, None]] = torch.randperm(used + 1, generator=c)[:used]
        s["block_table"], s["lengths"] = (t.to(torch.int32).cuda() for t in (table, lengths))
        s["first"] = (lengths - case["window"]).clamp(min=0).to(torch.int32).cuda() if case["window"] else None
        s["q"] = 2 * torch.randn((case["requests"], case["heads"] * case["head_dim"]), device="cuda", generator=g)
        return s
    n, k = case["rows"], case["width"]
    s["x"], s["y"] = (torch.randn((n, k), device="cuda", generator=g) for _ in range(2))
    s["y"] *= 3
    for side in ("post", "pre"):
        kind = case[side]
        s[side + "_weight"] = 1 + 0.1 * torch.randn(k, device="cuda", generator=g) if kind else None
        s[side + "_bias"] = 0.1 * torch.randn(k, device="cuda", generator=g) if kind == "layer" else None
    s["gate"] = None if not case["gate"] else torch.rand(
        (n, k) if case["gate"] == "token" else (k,), device="cuda", generator=g)
    return s


# ------------------------------------------------------------- plain forms
def _cdiv(a, b):
    return (a + b - 1) // b


def _plain_assign(s):
    page, rows = s["case"]["page"], s["case"]["rows"]
    old, table = s["lengths"].long(), s["block_table"].long()
    new = (old + s["delta"]).clamp(min=0)
    held, need = _cdiv(old, page)[:, None], _cdiv(new, page)[:, None]
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    # pages handed back, request by request, on top of the free list
    back = (j >= need) & (j < held)
    rank = back.flatten().cumsum(0).view_as(back) - 1
    cap, count = s["free_pages"].numel(), s["free_count"].long()
    at = torch.where(back, count + rank, cap)
    free = torch.cat([s["free_pages"].long(), table.new_zeros(1)])
    free = free.scatter(0, at.flatten(), table.flatten())[:cap]
    top = count + back.sum()
    # pages taken from the top, request by request
    take = (j >= held) & (j < need)
    rank = take.flatten().cumsum(0).view_as(take) - 1
    table = torch.where(take, free[(top - 1 - rank).clamp(min=0)], table)
    # one row per new token
    grown = (new - old).clamp(min=0)
    row_start = torch.cat([grown.new_zeros(1), grown.cumsum(0)])
    t = torch.arange(rows, device=table.device)
    valid = t < row_start[-1]
    request = torch.searchsorted(row_start[1:].contiguous(), t, right=True).clamp(max=old.numel() - 1)
    position = old[request] + t - row_start[request]
    where = (position // page).clamp(0, table.shape[1] - 1)
    slot = table[request, where] * page + position % page
    out = dict(lengths=new, free_count=top - take.sum(), block_table=table, free_pages=free,
               slots=torch.where(valid, slot, -1), positions=torch.where(valid, position, 0),
               requests=torch.where(valid, request, -1), row_start=row_start)
    return {k: v.to(torch.int32) for k, v in out.items()}


def _rotate(x, cos, sin, interleaved):
    """x [rows, heads, head_dim], its first 2 * cos.shape[1] columns rotated."""
    n = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
    else:
        a, b = x[..., :n], x[..., n:2 * n]
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], dim=-1).flatten(-2) if interleaved else torch.cat([u, v], dim=-1)
    return torch.cat([turned, x[..., 2 * n:]], dim=-1)


def _values(pool, scale):
    """What a pool of codes stands for."""
    return (pool.float() * scale[..., None]).to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    n, d = c["rows"], c["head_dim"]
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotate(s["q"].reshape(n, -1, d), cos, sin, c["interleaved"]).reshape(n, -1)
    k = _rotate(s["k_new"].reshape(n, -1, d), cos, sin, c["interleaved"])
    v = s["v_new"].reshape(n, -1, d)
    # padding rows repeat what row 0 writes
    row = torch.where(s["slots"] >= 0, torch.arange(n, device=q.device), 0)
    slot = s["slots"][row].long()
    out = [q]
    for name, x in (("k", k), ("v", v)):
        pool, x = s[name].view(-1, c["kv_heads"], d), x[row]
        if c["dtype"] == "i8":
            amax = x.abs().amax(dim=-1)
            code = (x * torch.where(amax > 0, 127.0 / amax, 0.0)[..., None]).round().clamp(-127, 127)
            pool[slot] = code.to(torch.int8)
            s[name + "_scale"].view(-1, c["kv_heads"])[slot] = amax / 127.0
            out.append(_values(s[name], s[name + "_scale"]))
        else:
            pool[slot] = x.to(pool.dtype)
            out.append(s[name])
    return out


def _plain_attention(s):
    c = s["case"]
    n, d, hk = c["requests"], c["head_dim"], c["kv_heads"]
    table = s["block_table"].long()
    q = s["q"].view(n, hk, -1, d) * d ** -0.5
    k, v = (s[name][table].flatten(1, 2).float() for name in ("k", "v"))
    if c["dtype"] == "i8":
        k, v = (x * s[name + "_scale"][table].flatten(1, 2)[..., None] for x, name in ((k, "k"), (v, "v")))
    j = torch.arange(k.shape[1], device=q.device)[None, :]
    seen = j < s["lengths"][:, None]
    if s["first"] is not None:
        seen = seen & (j >= s["first"][:, None])
    v = torch.where(seen[:, :, None, None], v, 0.0)
    score = torch.matmul(q, k.permute(0, 2, 3, 1))
    score = torch.where(seen[:, None, None, :], score, -math.inf)
    top = score.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    weight = torch.exp(score - top)
    total = weight.sum(dim=-1, keepdim=True)
    out = torch.matmul(weight, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return [out.reshape(n, -1), lse.reshape(n, -1)]


def _norm(x, kind, weight, bias):
    if not kind:
        return x
    if kind == "layer":
        x = x - x.mean(dim=-1, keepdim=True)
    x = x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * weight
    return x + bias if bias is not None else x


def _plain_norm(s):
    c = s["case"]
    t = _norm(s["y"], c["post"], s["post_weight"], s["post_bias"])
    t = t if s["gate"] is None else t * s["gate"]
    h = s["x"] + c["alpha"] * t
    n = _norm(h, c["pre"], s["pre_weight"], s["pre_bias"])
    if not c["codes"]:
        return [h, n]
    amax = n.abs().amax(dim=-1)
    code = (n * torch.where(amax > 0, 127.0 / amax, 0.0)[:, None]).round().clamp(-128, 127)
    return [h, _values(code, amax / 127.0), amax]


# --------------------------------------------------------- the framework's
def _own_assign(api, s):
    c = s["case"]
    a = api.kv_assign(s["lengths"], s["delta"], s["block_table"], s["free_pages"], s["free_count"],
                      c["page"], c["rows"])
    return dict(lengths=a.lengths, free_count=a.free_count, block_table=s["block_table"],
                free_pages=s["free_pages"], slots=a.slots, positions=a.positions,
                requests=a.requests, row_start=a.row_start)


def _cache(api, s):
    """The cache handle that a program keeps beside its pools."""
    if "cache" not in s:
        s["cache"] = api.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s["cache"]


def _own_append(api, s):
    q = api.rope_append(s["q"], s["k_new"], s["v_new"], s["positions"], s["slots"], _cache(api, s),
                        inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"])
    if s["case"]["dtype"] == "i8":
        return [q, _values(s["k"], s["k_scale"]), _values(s["v"], s["v_scale"])]
    return [q, s["k"], s["v"]]


def _own_attention(api, s):
    cache = _cache(api, s)
    if "workspace" not in s:   # kept beside the cache, as its users do
        s["workspace"] = api.paged_attention_workspace(s["case"]["requests"], s["case"]["heads"], cache)
    return list(api.paged_attention(s["q"], cache, s["block_table"], s["lengths"], first=s["first"],
                                    ws=s["workspace"], return_lse=True))


def _own_norm(api, s):
    c = s["case"]
    r = api.residual_norm(s["x"], s["y"], post=c["post"] or None, post_weight=s["post_weight"],
                          post_bias=s["post_bias"], gate=s["gate"], alpha=c["alpha"], pre=c["pre"],
                          pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], eps=EPS,
                          quantize=c["codes"])
    if not c["codes"]:
        return [r.h, r.n]
    return [r.h, _values(r.xq, r.amax / 127.0), r.amax]


def run(state):
    op = state["case"]["op"]
    if own:
        from ternary_weight_decoder_b200 import api
        return {"assign": _own_assign, "append": _own_append, "attention": _own_attention,
                "norm": _own_norm}[op](api, state)
    return {"assign": _plain_assign, "append": _plain_append, "attention": _plain_attention,
            "norm": _plain_norm}[op](state)


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "assign":
        # lengths, deltas and free list's end read; lengths, row starts, the
        # slots, positions and requests of every row, and the new pages written
        n = case["requests"]
        return {"bytes": 4 * (4 * n + 3 * case["rows"] + case["rows"] // case["page"]), "flops": 0}
    if op == "append":
        wide = case["kv_heads"] * case["head_dim"]
        size = 1 if case["dtype"] == "i8" else 2
        real = case["rows"] - case["pad"]
        b = case["rows"] * (8 * case["heads"] * case["head_dim"] + 8) + real * (8 * wide + 2 * size * wide)
        if size == 1:   # the scales, and the values that the codes stand for
            pool = (_cdiv(real, case["page"]) + 1) * case["page"] * wide
            b += real * 8 * case["kv_heads"] + 2 * 3 * pool
        return {"bytes": b, "flops": 3 * case["rows"] * case["rotary"] * (case["heads"] + case["kv_heads"])}
    if op == "attention":
        seen = [min(n, case["window"] or n) for n in _lengths(case)]
        wide = case["kv_heads"] * case["head_dim"]
        size = 1 if case["dtype"] == "i8" else 2
        b = sum(seen) * (2 * wide * size + (8 * case["kv_heads"] if size == 1 else 0))
        b += 4 * sum(_cdiv(n, case["page"]) for n in seen)
        b += case["requests"] * (8 * case["heads"] * case["head_dim"] + 4 * case["heads"] + 4)
        return {"bytes": b, "flops": 4 * sum(seen) * case["heads"] * case["head_dim"]}
    n = case["rows"] * case["width"]
    b = 16 * n + (4 * n if case["gate"] == "token" else 0)
    if case["codes"]:   # codes in place of 32-bit values, then the values they stand for
        b += -3 * n + 3 * n
    return {"bytes": b, "flops": 12 * n}


# ------------------------------------------------------------------- exact
def _exact_append(s):
    c = s["case"]
    n, half = c["rows"], c["rotary"] // 2
    phase = torch.polar(torch.ones(n, half, dtype=torch.float64, device="cuda"),
                        torch.outer(s["positions"].double(), s["inv_freq"]))

    def turn(x):
        x = x.double().reshape(n, -1, c["head_dim"]).clone()
        head = x[:, :, :2 * half]
        re, im = (head[:, :, 0::2], head[:, :, 1::2]) if c["interleaved"] else \
            (head[:, :, :half], head[:, :, half:])
        z = torch.complex(re.contiguous(), im.contiguous()) * phase.unsqueeze(1)
        re.copy_(z.real)
        im.copy_(z.imag)
        return x

    out = [turn(s["q"]).flatten(1)]
    real = n - c["pad"]
    at = s["slots"][:real].long()
    for name, x in (("k", turn(s["k_new"])), ("v", s["v_new"].double().reshape(n, -1, c["head_dim"]))):
        pool = s[name].double()
        if c["dtype"] == "i8":
            pool *= s[name + "_scale"].double().unsqueeze(-1)
            step = x.abs().max(dim=-1, keepdim=True).values / 127
            x = torch.where(step > 0, torch.round(x / step) * step, x)
        pool.view(-1, c["kv_heads"], c["head_dim"]).index_copy_(0, at, x[:real])
        out.append(pool)
    return out


def _exact_attention(s):
    c = s["case"]
    n, d, group = c["requests"], c["head_dim"], c["heads"] // c["kv_heads"]
    out = torch.zeros(n, c["heads"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, c["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    lengths = s["lengths"].tolist()
    firsts = [0] * n if s["first"] is None else s["first"].tolist()
    for r in range(n):
        lo, hi = firsts[r], lengths[r]
        if hi <= lo:
            continue
        at = torch.arange(lo, hi, device="cuda")
        page, offset = s["block_table"][r].long()[at // c["page"]], at % c["page"]
        rows = {}
        for name in ("k", "v"):
            x = s[name][page, offset].double()
            if c["dtype"] == "i8":
                x = x * s[name + "_scale"][page, offset].double().unsqueeze(-1)
            rows[name] = x
        for h in range(c["heads"]):
            z = rows["k"][:, h // group] @ s["q"][r, h * d:(h + 1) * d].double() / math.sqrt(d)
            lse[r, h] = torch.logsumexp(z, dim=0)
            out[r, h] = torch.exp(z - lse[r, h]) @ rows["v"][:, h // group]
    return [out.view(n, -1), lse]


def _exact_norm(s):
    c = s["case"]

    def normed(x, side):
        if not c[side]:
            return x
        if c[side] == "layer":
            var, mean = torch.var_mean(x, dim=1, keepdim=True, correction=0)
            x = (x - mean) * torch.rsqrt(var + EPS)
        else:
            x = x * torch.rsqrt(x.square().sum(dim=1, keepdim=True) / c["width"] + EPS)
        x = x * s[side + "_weight"].double()
        return x if s[side + "_bias"] is None else x + s[side + "_bias"].double()

    t = normed(s["y"].double(), "post")
    if s["gate"] is not None:
        t = t * s["gate"].double()
    h = torch.add(s["x"].double(), t, alpha=c["alpha"])
    n = normed(h, "pre")
    if not c["codes"]:
        return [h, n]
    amax = n.abs().max(dim=1).values
    step = (amax / 127).unsqueeze(1)
    return [h, torch.where(step > 0, torch.round(n / step) * step, n), amax]


def exact(case, seed):
    if case["op"] == "assign":   # whole numbers alone
        return None
    return {"append": _exact_append, "attention": _exact_attention,
            "norm": _exact_norm}[case["op"]](prepare(case, seed))
