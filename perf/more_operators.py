"""Cases of a speculative decode step over a paged cache: appending rotated keys and values to pages of 16, 8 or
4 bits, reading pages back as rows, attention of the newest tokens over 4-bit pages, and the verification
of drafted tokens against the target's probabilities.

`run` with `own` false computes an operator in its plain form, elementary torch operations in 32 bits (64 for
angles and sums of probabilities) that are rounded once at the end; with `own` true it makes the calls a program
makes of the package. Both take what `prepare` gives. `exact` is the definition in 64 bits, written apart.

4-bit pages hold E2M1 codes, two to a byte, and an E4M3 scale for each 16 dims of a row. Stored byte (dim / 8) t + 2 s + i
of a key's row is its byte 8 s + 2 t + i (dims 2 b, 2 b + 1 in byte b), stored byte (dim / 16) r + s of a value's row
its byte 8 s + r.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1, "e2m1": 0.5625}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
THETA = 160000.0


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a batch of 64: a token of each request is rotated and joins its bf16 pages
        dict(name="append step 64x1", op="append", batch=64, most=64, each=True, heads=8, group=4, dim=128, page=64,
             type="bf16", cache="bf16", context=500, rotary=128, pairs="halves", shape=1),
        # a packed batch of prompts, 65,536 tokens in 7 requests, into FP8 pages
        dict(name="append prompt 65536 fp8", op="append", batch=7, most=65536, each=False, heads=8, group=4, dim=128, page=64,
             type="bf16", cache="e4m3", context=0, rotary=128, pairs="halves", shape=2),
        # chunks of prompts behind contexts in 4-bit pages, half of each head rotated; the chunks' attention then
        # takes the contexts as rows
        dict(name="append chunk fp4 500", op="append", batch=5, most=500, each=False, heads=4, group=6, dim=128, page=16,
             type="f16", cache="e2m1", context=4000, rotary=64, pairs="neighbours", shape=3),
        # rows of a prefix kept in FP8 pages of small heads, for the attention of a chunk behind it
        dict(name="read fp8 3x2500", op="read", batch=3, most=2500, heads=4, dim=64, page=16, type="f16", cache="e4m3", shape=4),
        # four long contexts out of 4-bit pages
        dict(name="read fp4 4x65536", op="read", batch=4, most=65536, heads=8, dim=128, page=128, type="bf16", cache="e2m1",
             shape=5),
        # one user's chat at a thousand tokens: nothing but latency
        dict(name="decode fp4 1x1000", op="decode", batch=1, queries=1, heads=8, group=4, dim=128, page=16, type="bf16",
             context=1000, ragged=False, window=0, shape=6),
        # an ordinary serving batch with contexts of any length up to 8,192
        dict(name="decode fp4 32x8192 ragged", op="decode", batch=32, queries=1, heads=8, group=8, dim=128, page=64,
             type="bf16", context=8192, ragged=True, window=0, shape=7),
        # drafts of five tokens for 64 requests, seven query heads to a key head
        dict(name="decode fp4 64x5x4097", op="decode", batch=64, queries=5, heads=4, group=7, dim=128, page=32, type="f16",
             context=4097, ragged=True, window=0, shape=8),
        # four requests at 131,072 positions
        dict(name="decode fp4 4x131072", op="decode", batch=4, queries=1, heads=8, group=8, dim=128, page=128,
             type="bf16", context=131072, ragged=False, window=0, shape=9),
        # one user's draft of four tokens
        dict(name="verify 1x5x131072", op="verify", batch=1, queries=5, vocabulary=131072, type="f32", drafter=True, ragged=False,
             shape=10),
        # drafts of four tokens for 64 requests
        dict(name="verify 64x5x131072", op="verify", batch=64, queries=5, vocabulary=131072, type="f32", drafter=True, ragged=False,
             shape=11),
        # drafts of up to seven tokens found by lookup in the text, over an odd vocabulary in 16 bits
        dict(name="verify 37x8x50001 lookup", op="verify", batch=37, queries=8, vocabulary=50001, type="bf16", drafter=False,
             ragged=True, shape=12),
    ]


def spread(rng, lo, hi):
    """A whole number of lo..hi, uniform in its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))))


def draw(rng):
    op = rng.choice(("append", "append", "read", "decode", "decode", "decode", "verify"))
    shape, dim = rng.randrange(1 << 30), rng.choice((64, 128))
    kind = rng.choice(("bf16", "f16"))
    page = 16 * rng.choice((1, 2, 3, 4, 5, 8, 16))
    heads = spread(rng, 1, 16)
    if op == "append":
        group, cache = spread(rng, 1, 16), rng.choice((kind, "e4m3", "e2m1"))
        most = spread(rng, 1, min(65536, 65536 * 8 * 6 * 128 // (heads * (group + 2) * dim)) if cache != "e2m1" else 500)
        batch = spread(rng, 1, min(128, most))
        return dict(op=op, batch=batch, most=most, each=False, heads=heads, group=group, dim=dim, page=page, type=kind, cache=cache,
                    context=rng.choice((0, spread(rng, 1, 4000))), rotary=32 * rng.randint(1, dim // 32),
                    pairs=rng.choice(("halves", "neighbours")), shape=shape)
    if op == "read":
        batch = spread(rng, 1, 64)
        return dict(op=op, batch=batch, most=spread(rng, 1, max(1, min(65536, 4 * 65536 * 8 * 128 // (batch * heads * dim)))), heads=heads,
                    dim=dim, page=page, type=kind, cache=rng.choice((kind, "e4m3", "e2m1")), shape=shape)
    if op == "decode":
        group, queries, batch = spread(rng, 1, 16), rng.choice((1, 1, 1, 2, 3, 5, 8)), spread(rng, 1, 128)
        room = 4 * 131072 * 8 * 128 // (batch * heads * dim)                   # at most the largest listed case's bytes
        room = min(room, 64 * 32768 * 64 // (batch * heads * group * queries))  # and a plain form that fits
        return dict(op=op, batch=batch, queries=queries, heads=heads, group=group, dim=dim, page=page, type=kind,
                    context=spread(rng, 1, max(1, min(131072, room))), ragged=rng.random() < 0.7,
                    window=rng.choice((0, 0, 0, spread(rng, 1, 1000))), shape=shape)
    queries, vocabulary = rng.choice((1, 2, 3, 4, 5, 6, 8)), spread(rng, 1000, 200000)
    return dict(op=op, batch=spread(rng, 1, max(1, min(128, 64 * 5 * 131072 // (queries * vocabulary)))), queries=queries, vocabulary=vocabulary,
                type=rng.choice(("f32", "f32", "bf16", "f16")), drafter=rng.random() < 0.7, ragged=rng.random() < 0.5, shape=shape)


def parts(case):
    """The tokens that each request of a packed batch brings (append) or has (read)."""
    n, total = case["batch"], case["most"]
    rng = random.Random(case["shape"])
    if case["op"] == "read":
        return [rng.randint(max(1, total // 2), total) for _ in range(n)]
    if case["each"]:
        return [total // n] * n
    cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def pasts(case):
    """The positions that each request has before its new tokens."""
    rng = random.Random(case["shape"] + 1)
    return [rng.randrange(case["context"] + 1) if case["op"] == "append" and case["context"] else 0 for _ in range(case["batch"])]


def visible(case):
    """Visible lengths [request][query] of a decode case: the newest query sees the whole context."""
    rng = random.Random(case["shape"])
    ends = [rng.randint(max(1, case["context"] // 50), case["context"]) if case["ragged"] else case["context"]
            for _ in range(case["batch"])]
    return [[max(0, e - case["queries"] + 1 + i) for i in range(case["queries"])] for e in ends]


def drafts(case):
    """The drafted tokens of each request of a verify case."""
    rng = random.Random(case["shape"])
    return [rng.randrange(case["queries"]) if case["ragged"] else case["queries"] - 1 for _ in range(case["batch"])]


def work(case):
    op = case["op"]
    if op == "verify":
        # a row of the target for each request, and one of the drafter's where a token is turned down (three in four)
        rows = case["batch"] * (1.75 if case["drafter"] else 1.0)
        return {"bytes": rows * case["vocabulary"] * SIZE[case["type"]] + case["batch"] * case["queries"] * 24, "flops": 0}
    dim, heads = case["dim"], case["heads"]
    if op == "append":
        new, row = sum(parts(case)), heads * dim
        total = 2 * new * row * (2 + SIZE[case["cache"]]) + 4 * new * row * case["group"]
        if case["cache"] == "e2m1":
            total += 2 * (new + sum(pasts(case))) * row * (2 + SIZE["e2m1"])
        return {"bytes": total, "flops": 3 * new * row * (1 + case["group"])}
    if op == "read":
        return {"bytes": 2 * sum(parts(case)) * heads * dim * (2 + SIZE[case["cache"]]), "flops": 0}
    low = (lambda e: max(0, e - case["window"])) if case["window"] else (lambda e: 0)
    vis = visible(case)
    held = sum(max(r) - low(min(r)) for r in vis)
    seen = sum(e - low(e) for r in vis for e in r)
    rows = case["batch"] * case["queries"] * heads * case["group"]
    return {"bytes": 2 * held * heads * dim * SIZE["e2m1"] + 2 * rows * dim * 2 + rows * 4, "flops": 4 * seen * heads * case["group"] * dim}


# ------------------------------------------------------------------------------------ 4-bit rows
def scales_for(x):
    """x [...][dims] -> for each 16 dims the smallest E4M3 value s with 6 s >= their largest magnitude, at least 2^-9."""
    t = x.reshape(*x.shape[:-1], -1, 16).abs().amax(-1).double() / 6
    step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
    return (torch.ceil(t / step) * step).clamp(min=2.0 ** -9, max=448.0)


def codes_for(x, s):
    """E2M1 codes of x / s, ties to the even code, -0 as 0."""
    y = (x.reshape(*x.shape[:-1], -1, 16) / s[..., None]).reshape(x.shape)
    a, c = y.abs(), torch.zeros(x.shape, dtype=torch.uint8, device=x.device)
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (a >= border) if up else (a > border)
    return c + 8 * ((y < 0) & (c > 0)).to(torch.uint8)


def stored(codes, keys):
    """Codes [...][dims] -> bytes [...][dims / 2] in the order of the pages."""
    b = codes[..., 0::2] | codes[..., 1::2] << 4
    lead, n = b.shape[:-1], b.shape[-1] // 8
    return (b.view(*lead, n, 4, 2).transpose(-3, -2) if keys else b.view(*lead, n, 8).transpose(-2, -1)).reshape(*lead, 8 * n)


def values(pool, scales, keys):
    """The values that bytes [...][dims / 2] and scales [...][dims / 16] stand for, in 32 bits (exactly)."""
    lead, n = pool.shape[:-1], pool.shape[-1] // 8
    b = (pool.reshape(*lead, 4, n, 2).transpose(-3, -2) if keys else pool.reshape(*lead, 8, n).transpose(-2, -1)).reshape(*lead, 8 * n)
    table = torch.tensor([*LEVELS, *(-x for x in LEVELS)], device=pool.device)
    x = torch.stack((table[(b & 15).int()], table[(b >> 4).int()]), -1).reshape(*lead, n, 16)
    return (x * scales.float()[..., None]).reshape(*lead, 16 * n)


# --------------------------------------------------------------------------------------- inputs
def pages_of(case, longest, g):
    """Pools of pages with values in every place, and tables that map each request's positions to pages in any order."""
    batch, page, heads, dim = case["batch"], case["page"], case["heads"], case["dim"]
    need = [-(-n // page) for n in longest]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((batch, max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    kind, pools, scales = case.get("cache", "e2m1"), [], []
    some = max(1, (1 << 26) // (heads * page * dim))
    for keys in (True, False):
        if kind == "e2m1":
            pool = torch.empty(total, heads, page, dim // 2, dtype=torch.uint8, device="cuda")
            scale = torch.empty(total, heads, page, dim // 16, dtype=TYPES["e4m3"], device="cuda")
        else:
            pool, scale = torch.empty(total, heads, page, dim, dtype=TYPES[kind], device="cuda"), None
        for lo in range(0, total, some):
            x = torch.randn(min(some, total - lo), heads, page, dim, generator=g, device="cuda")
            if kind == "e2m1":
                s = scales_for(x)
                pool[lo:lo + some] = stored(codes_for(x, s.float()), keys)
                scale[lo:lo + some] = s.to(scale.dtype)
            else:
                pool[lo:lo + some] = x.to(pool.dtype)
        pools.append(pool)
        scales.append(scale)
    return dict(k_pages=pools[0], v_pages=pools[1], k_s=scales[0], v_s=scales[1], table=table)


def starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "verify":
        return prepare_verify(case, g, s)
    dim, heads, kind = case["dim"], case["heads"], TYPES[case["type"]]

    def normal(*shape, by=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * by).to(kind)

    s["k_scale"], s["v_scale"] = 1.0, 1.0
    if case["op"] == "append":
        new, past = parts(case), pasts(case)
        both = [a + b for a, b in zip(new, past)]
        s.update(pages_of(case, both, g))
        # queries, keys and values as one projection leaves them: interleaved rows of one buffer
        rows = normal(sum(new), heads * (case["group"] + 2), dim)
        s["q"], s["k"], s["v"] = rows.split((heads * case["group"], heads, heads), 1)
        s["q_out"] = torch.empty(sum(new), heads * case["group"], dim, dtype=kind, device="cuda")
        s["cu"], s["start"] = starts(new), torch.tensor(past, dtype=torch.int64, device="cuda")
        half = torch.arange(case["rotary"] // 2, dtype=torch.float64)
        s["inv_freq"] = (THETA ** (-2.0 * half / case["rotary"])).float().cuda()
        if case["cache"] == "e4m3":
            s["k_scale"], s["v_scale"] = 0.03125, 0.0234375
        if case["cache"] == "e2m1":
            s["k_scale"], s["v_scale"] = 0.125, 0.09375
            s["cu_all"] = starts(both)
            s["k_rows"], s["v_rows"] = (torch.empty(sum(both), heads, dim, dtype=kind, device="cuda") for _ in range(2))
    elif case["op"] == "read":
        n = parts(case)
        s.update(pages_of(case, n, g))
        s["cu_all"] = starts(n)
        s["k_rows"], s["v_rows"] = (torch.empty(sum(n), heads, dim, dtype=kind, device="cuda") for _ in range(2))
        if case["cache"] in ("e4m3", "e2m1"):
            s["k_scale"], s["v_scale"] = 0.75, 1.25
    else:
        vis = visible(case)
        s["longest"] = max(max(r) for r in vis)
        s.update(pages_of(case, [max(r) for r in vis], g))
        s["vis"] = torch.tensor(vis, dtype=torch.int32, device="cuda")
        s["q"] = normal(case["batch"], case["queries"], heads * case["group"], dim, by=2.0)
        s["k_scale"], s["v_scale"] = 0.75, 1.25
        s["scale"] = 1.0 / math.sqrt(dim)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:-1], dtype=torch.float32, device="cuda")
    if own:
        import hierarchical_sparse_attention_index_gb300 as H
        s["cache"] = H.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["k_scale"], s["v_scale"], s["k_s"], s["v_s"])
        if case["op"] == "decode":
            s["ws"] = H.new_paged_workspace(s["cache"], heads * case["group"], case["queries"], s["longest"])
    return s


def prepare_verify(case, g, s):
    batch, nq, n = case["batch"], case["queries"], case["vocabulary"]
    logits = torch.randn(batch, nq, n, generator=g, device="cuda") * 2.5
    s["p"] = torch.softmax(logits, -1).to(TYPES[case["type"]])
    guess = logits[:, :-1] + 0.7 * torch.randn(batch, nq - 1, n, generator=g, device="cuda")
    # drafted by chance from the drafter's own probabilities; a lookup takes likely tokens and gives none
    noise = -torch.log(-torch.log(torch.rand(guess.shape, generator=g, device="cuda").clamp(1e-30, 1 - 1e-7)))
    s["drafted"] = (guess + noise * (1.0 if case["drafter"] else 0.2)).argmax(-1).to(torch.int32) if nq > 1 else \
        torch.empty(batch, 0, dtype=torch.int32, device="cuda")
    s["q"] = torch.softmax(guess, -1).to(TYPES[case["type"]]) if case["drafter"] else None
    s["u_accept"] = torch.rand(batch, nq - 1, generator=g, device="cuda")
    s["u_sample"] = torch.rand(batch, generator=g, device="cuda")
    s["n_draft"] = torch.tensor(drafts(case), dtype=torch.int32, device="cuda")
    s["accepted"] = torch.empty(batch, dtype=torch.int32, device="cuda")
    s["tokens"] = torch.empty(batch, nq, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        import hierarchical_sparse_attention_index_gb300 as H
        if case["op"] == "verify":
            H.hsa_draft_verify(s["p"], s["q"], s["drafted"], s["u_accept"], s["u_sample"], s["accepted"], s["tokens"],
                               n_draft=s["n_draft"])
            return s["accepted"], s["tokens"]
        if case["op"] == "decode":
            H.hsa_paged_attn_decode(s["cache"], s["q"], s["vis"], s["longest"], s["scale"], s["out"], s["ws"],
                                    window=case["window"], lse=s["lse"])
            return s["out"], s["lse"]
        if case["op"] == "append":
            H.hsa_paged_cache_append(s["cache"], s["k"], s["v"], s["inv_freq"], q=s["q"], q_out=s["q_out"], cu=s["cu"],
                                     start=s["start"], pairs=H.HSA_ROPE_HALVES if case["pairs"] == "halves" else H.HSA_ROPE_NEIGHBOURS)
            if case["cache"] != "e2m1":
                return s["q_out"], s["k_pages"], s["v_pages"]
        H.hsa_paged_cache_read(s["cache"], s["k_rows"], s["v_rows"], cu=s["cu_all"])
        return (s["q_out"], s["k_rows"], s["v_rows"]) if case["op"] == "append" else (s["k_rows"], s["v_rows"])
    return {"verify": plain_verify, "decode": plain_decode, "append": plain_append, "read": plain_read}[case["op"]](s)


def places(s, cu, start):
    """Page and row in it of each packed row."""
    cu, page = cu.long(), s["case"]["page"]
    t = torch.arange(int(s["rows"]), device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    at = t - cu[b] + (start[b] if start is not None else 0)
    return s["table"][b, at // page].long(), at % page, at


def plain_append(s):
    case = s["case"]
    kind, r = TYPES[case["type"]], case["rotary"]
    s["rows"] = s["k"].shape[0]
    where, row, at = places(s, s["cu"], s["start"])
    angle = at.double()[:, None] * s["inv_freq"].double()
    c, n = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotated(x):
        x = x.float()
        if case["pairs"] == "halves":
            a, b = x[..., :r // 2], x[..., r // 2:r]
            return torch.cat((a * c - b * n, a * n + b * c, x[..., r:]), -1)
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        return torch.cat((torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2), x[..., r:]), -1)

    s["q_out"].copy_(rotated(s["q"]))
    for pool, scales, x, scale, keys in ((s["k_pages"], s["k_s"], rotated(s["k"]), s["k_scale"], True),
                                         (s["v_pages"], s["v_s"], s["v"].float(), s["v_scale"], False)):
        if case["cache"] == "e2m1":
            x = x * (1.0 / scale)
            group = scales_for(x)
            pool[where, :, row] = stored(codes_for(x, group.float()), keys)
            scales.view(torch.uint8)[where, :, row] = group.to(scales.dtype).view(torch.uint8)
        elif case["cache"] == "e4m3":
            pool.view(torch.uint8)[where, :, row] = (x / scale).clamp(-448, 448).to(pool.dtype).view(torch.uint8)
        else:
            pool[where, :, row] = x.to(kind)
    if case["cache"] != "e2m1":
        return s["q_out"], s["k_pages"], s["v_pages"]
    return (s["q_out"], *plain_read(s))


def plain_read(s):
    s["rows"] = s["k_rows"].shape[0]
    where, row, _ = places(s, s["cu_all"], None)
    for pool, scales, out, scale, keys in ((s["k_pages"], s["k_s"], s["k_rows"], s["k_scale"], True),
                                           (s["v_pages"], s["v_s"], s["v_rows"], s["v_scale"], False)):
        if scales is not None:
            x = values(pool[where, :, row], scales.view(torch.uint8)[where, :, row].view(scales.dtype), keys)
        elif pool.element_size() == 1:
            x = pool.view(torch.uint8)[where, :, row].view(pool.dtype).float()
        else:
            x = pool[where, :, row].float()
        out.copy_(x * scale)
    return s["k_rows"], s["v_rows"]


def plain_decode(s):
    case = s["case"]
    batch, heads, dim, nq = case["batch"], case["heads"], case["dim"], case["queries"]
    where = s["table"].clamp(min=0).long()
    k, v = (values(p[where], c.view(torch.uint8)[where].view(c.dtype), keys).transpose(2, 3).reshape(batch, -1, heads, dim)
            for p, c, keys in ((s["k_pages"], s["k_s"], True), (s["v_pages"], s["v_s"], False)))   # [b][position][head][dim]
    vis = s["vis"].long()[:, :, None]
    at = torch.arange(k.shape[1], device="cuda")
    seen = at < vis
    if case["window"]:
        seen &= at >= vis - case["window"]
    q = s["q"].float().view(batch, nq, heads, case["group"], dim)
    x = torch.einsum("bihgd,bthd->bihgt", q, k) * (s["scale"] * s["k_scale"])
    x = x.masked_fill(~seen[:, :, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("bihgt,bthd->bihgd", p, v) * s["v_scale"] / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + top)[..., 0]
    return o.to(s["q"].dtype).reshape(s["q"].shape), lse.reshape(s["lse"].shape)


def plain_verify(s):
    case = s["case"]
    batch, nq, drafted = case["batch"], case["queries"], s["drafted"].long()
    row, place, n = torch.arange(batch, device="cuda"), torch.arange(nq, device="cuda"), s["n_draft"].long()
    if nq > 1:
        p_x = s["p"][:, :-1].gather(2, drafted[..., None])[..., 0].double()
        q_x = s["q"].gather(2, drafted[..., None])[..., 0].double() if s["q"] is not None else 1.0
        take = (s["u_accept"].double() * q_x < p_x) & (place[:-1] < n[:, None])
        kept = take.long().cumprod(1).sum(1)
    else:
        kept = torch.zeros_like(n)
    w = s["p"][row, kept].double()
    if nq > 1:
        turned, at = kept < n, kept.clamp(max=nq - 2)
        if s["q"] is not None:
            w = torch.where(turned[:, None], w - s["q"][row, at].double(), w).clamp(min=0)
        else:
            w[row[turned], drafted[row, at][turned]] = 0
    sums = w.cumsum(-1)
    token = (sums <= s["u_sample"].double()[:, None] * sums[:, -1:]).sum(1)
    tokens = torch.where(place < kept[:, None], torch.cat((drafted, drafted.new_zeros(batch, 1)), 1), -1)
    tokens[row, kept] = token
    s["accepted"].copy_(kept)
    s["tokens"].copy_(tokens)
    return s["accepted"], s["tokens"]


# ------------------------------------------------------------------------- the definition, 64 bits
def to_e4m3(x):
    """The nearest E4M3 value of each element (ties to the even one), beyond 448 the border."""
    size = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(size.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(size / step) * step).clamp(max=448.0)


def to_e2m1(x):
    """x [...][dims] as 4-bit pages hold it: a scale for each 16 dims, nearest levels, ties to the even one."""
    y = x.reshape(-1, 16)
    amax = y.abs().amax(1, keepdim=True)
    grid = torch.tensor(sorted({m * 2.0 ** e for m in range(8, 16) for e in range(-9, 6)} | {m * 2.0 ** -9 for m in range(1, 8)}),
                        dtype=torch.float64, device=x.device)
    grid = grid[grid <= 448]
    s = grid[torch.searchsorted(grid, (amax / 6).contiguous()).clamp(max=grid.numel() - 1)]
    size = (y / s).abs().clamp(max=6.0)
    step = torch.exp2(torch.floor(torch.log2(size.clamp(min=1.0))) - 1)
    return (torch.sign(y) * torch.round(size / step) * step * s).reshape(x.shape)


def read_pages(s, b, n):
    """The first n positions of request b as [n][heads][dim] in 64 bits."""
    page, got = s["case"]["page"], []
    where = s["table"][b, :-(-n // page)].long()
    for pool, scales, scale, keys in ((s["k_pages"], s["k_s"], s["k_scale"], True), (s["v_pages"], s["v_s"], s["v_scale"], False)):
        if scales is not None:
            half, m = pool.shape[-1], pool.shape[-1] // 8
            order = [m * 2 * t + 2 * g + i if keys else m * (2 * t + i) + g for g in range(m) for t in range(4) for i in range(2)]
            b8 = pool[where][..., torch.tensor(order, device="cuda")].long()
            c = torch.stack((b8 & 15, b8 >> 4), -1).flatten(-2)
            e, f = (c >> 1 & 3).double(), (c & 1).double()
            x = torch.where(e > 0, torch.exp2(e - 1) * (1 + f / 2), f / 2) * (1 - 2 * (c >> 3)).double()
            x = x * scales.view(torch.uint8)[where].view(scales.dtype).double().repeat_interleave(16, -1)
            assert x.shape[-1] == 2 * half
        else:
            x = (pool.view(torch.uint8)[where].view(pool.dtype) if pool.element_size() == 1 else pool[where]).double()
        got.append(x.transpose(1, 2).flatten(0, 1)[:n] * scale)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return {"verify": exact_verify, "decode": exact_decode, "append": exact_append, "read": exact_read}[case["op"]](s)


def exact_read(s):
    both = [read_pages(s, b, n) for b, n in enumerate(parts(s["case"])) if n]
    return tuple(torch.cat(x) for x in zip(*both))


def exact_append(s):
    case, r = s["case"], s["case"]["rotary"]
    new, past = parts(case), pasts(case)
    four = case["cache"] == "e2m1"
    pools = None if four else [s["k_pages"].double(), s["v_pages"].double()]
    q_out, rows = [], ([], [])
    t0 = 0

    def turn(x, at):
        x = x.double().clone()
        angle = at.double()[:, None] * s["inv_freq"].double()
        by = torch.polar(torch.ones_like(angle), angle)[:, None]
        if case["pairs"] == "halves":
            z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * by
            x[..., :r] = torch.cat((z.real, z.imag), -1)
        else:
            x[..., :r] = torch.view_as_real(torch.view_as_complex(x[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * by).flatten(-2)
        return x

    for b, (n, old) in enumerate(zip(new, past)):
        at = torch.arange(old, old + n, device="cuda")
        mine = slice(t0, t0 + n)
        t0 += n
        q_out.append(turn(s["q"][mine], at))
        before = read_pages(s, b, old) if four else None
        for i, (x, scale) in enumerate(((turn(s["k"][mine], at), s["k_scale"]), (s["v"][mine].double(), s["v_scale"]))):
            if four:
                rows[i].append(torch.cat((before[i], to_e2m1(x / scale) * scale if n else x)))
            else:
                pools[i][s["table"][b].long()[at // case["page"]], :, at % case["page"]] = to_e4m3(x / scale) if case["cache"] == "e4m3" else x
    return (torch.cat(q_out), *(torch.cat(x) for x in rows)) if four else (torch.cat(q_out), *pools)


def exact_decode(s):
    case = s["case"]
    dim, heads, group, w = case["dim"], case["heads"], case["group"], case["window"] or 1 << 40
    if sum(max(r) for r in visible(case)) * heads * group * case["queries"] > 1 << 32:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for b, ends in enumerate(visible(case)):
        n = max(ends)
        if not n:
            continue
        k, v = read_pages(s, b, n)
        ends = torch.tensor(ends, device="cuda")
        at = torch.arange(n, device="cuda")[None, :]
        hide = (at >= ends[:, None]) | (at < ends[:, None] - w)
        for h in range(heads):
            mine = slice(h * group, (h + 1) * group)
            x = (s["q"][b, :, mine].double().reshape(-1, dim) @ k[:, h].T).view(-1, group, n) * s["scale"]
            x.masked_fill_(hide[:, None, :], -math.inf)
            l = torch.logsumexp(x, -1)
            p = (x - l[..., None]).exp().nan_to_num_(nan=0.0)          # a query that sees no key has the output 0
            out[b, :, mine], lse[b, :, mine] = (p.view(-1, n) @ v[:, h]).view(-1, group, dim), l
    return out, lse


def exact_verify(s):
    case, accepted, tokens = s["case"], [], []
    p, drafted, u = s["p"], s["drafted"].tolist(), s["u_accept"].tolist()
    for b, n in enumerate(drafts(case)):
        kept = 0
        while kept < n:
            x = drafted[b][kept]
            if not u[b][kept] * (float(s["q"][b, kept, x]) if s["q"] is not None else 1.0) < float(p[b, kept, x]):
                break
            kept += 1
        w = p[b, kept].double()
        if kept < n:
            taken = s["q"][b, kept].double() if s["q"] is not None else torch.zeros_like(w).index_fill_(0, torch.tensor(drafted[b][kept], device="cuda"), 2.0)
            w = torch.relu(w - taken)
        sums = torch.cumsum(w, 0)
        token = int(torch.searchsorted(sums, (sums[-1] * float(s["u_sample"][b])).reshape(1), right=True))
        accepted.append(kept)
        tokens.append(drafted[b][:kept] + [token] + [-1] * (case["queries"] - kept - 1))
    return (torch.tensor(accepted, dtype=torch.int32, device="cuda"), torch.tensor(tokens, dtype=torch.int32, device="cuda"))
