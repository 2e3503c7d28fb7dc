"""Cases of the dense attention operators: writing keys and values into a paged cache, attention
of the newest tokens over that cache, and causal attention over packed prompts.

`run` with `own` false computes an operator in its plain form, elementary torch operations in 32
bits that are rounded once at the end; with `own` true it makes the call a program makes of the
package. Both take what `prepare` gives. `exact` is the definition in 64 bits, written apart.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "e4m3": 1}


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a batch of 64: a single token of each request joins its pages
        dict(name="write step 64x1", op="write", batch=64, most=1, ragged=False, heads=8, dim=128, page=64,
             type="bf16", cache="bf16", context=500, shape=1),
        # a whole prompt of a packed batch, 65,536 tokens in 7 requests
        dict(name="write prompt 65536", op="write", batch=7, most=65536, ragged=True, heads=8, dim=128, page=64,
             type="bf16", cache="bf16", context=0, shape=2),
        # a chunk of a packed batch appended to FP8 pages, an odd number of tokens
        dict(name="write chunk fp8 12345", op="write", batch=5, most=12345, ragged=True, heads=4, dim=64, page=16,
             type="f16", cache="e4m3", context=300, shape=3),
        # one user's chat at a thousand tokens: nothing but latency
        dict(name="decode 1x1000", op="decode", batch=1, queries=1, heads=8, group=4, dim=128, page=16, type="bf16",
             cache="bf16", context=1000, ragged=False, window=0, shape=4),
        # an ordinary serving batch with contexts of any length up to 8,192
        dict(name="decode 32x8192 ragged", op="decode", batch=32, queries=1, heads=8, group=8, dim=128, page=64,
             type="bf16", cache="bf16", context=8192, ragged=True, window=0, shape=5),
        # verifying a draft of five tokens for 64 requests, seven query heads to a key head
        dict(name="verify 64x5x4097", op="decode", batch=64, queries=5, heads=4, group=7, dim=128, page=32, type="f16",
             cache="f16", context=4097, ragged=True, window=0, shape=6),
        # four requests at 131,072 positions over FP8 pages: the largest read
        dict(name="decode fp8 4x131072", op="decode", batch=4, queries=1, heads=8, group=8, dim=128, page=128,
             type="bf16", cache="e4m3", context=131072, ragged=False, window=0, shape=7),
        # one short prompt
        dict(name="prompt 1x77", op="prompt", batch=1, most=77, past=0, heads=8, group=4, dim=128, type="bf16",
             window=0, ragged=False, shape=8),
        # a packed batch of prompts of different lengths
        dict(name="prompt packed 16381", op="prompt", batch=12, most=16381, past=0, heads=8, group=8, dim=128,
             type="bf16", window=0, ragged=True, shape=9),
        # one long document
        dict(name="prompt 1x16384", op="prompt", batch=1, most=16384, past=0, heads=4, group=8, dim=128, type="bf16",
             window=0, ragged=False, shape=10),
        # chunks of prompts behind a context that is already there
        dict(name="prompt chunk 4096 past", op="prompt", batch=6, most=3000, past=4096, heads=4, group=6, dim=64,
             type="f16", window=0, ragged=True, shape=11),
        # a layer with a sliding window of 128 over packed prompts
        dict(name="prompt window 32768", op="prompt", batch=9, most=32768, past=0, heads=8, group=8, dim=64,
             type="bf16", window=128, ragged=True, shape=12),
    ]


def spread(rng, lo, hi):
    """A whole number of lo..hi, uniform in its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))))


def draw(rng):
    op = rng.choice(("write", "decode", "decode", "prompt", "prompt"))
    shape, dim = rng.randrange(1 << 30), rng.choice((64, 128))
    kind = rng.choice(("bf16", "f16"))
    page = 16 * rng.choice((1, 2, 3, 4, 5, 8, 16))
    if op == "write":
        heads = spread(rng, 1, 16)
        most = spread(rng, 1, min(65536, 65536 * 8 * 128 // (heads * dim)))
        return dict(op=op, batch=spread(rng, 1, min(128, most)), most=most, ragged=True, heads=heads, dim=dim, page=page,
                    type=kind, cache=rng.choice((kind, kind, "e4m3")), context=rng.choice((0, spread(rng, 1, 700))),
                    shape=shape)
    if op == "decode":
        heads, group, queries = spread(rng, 1, 16), spread(rng, 1, 16), rng.choice((1, 1, 1, 2, 3, 5, 8))
        cache = rng.choice((kind, kind, "e4m3"))
        batch = spread(rng, 1, 128)
        room = 4 * 131072 * 8 * 128 // (batch * heads * dim * SIZE[cache])     # at most the largest listed case's bytes
        room = min(room, 64 * 32768 * 64 // (batch * heads * group * queries))  # and a plain form that fits
        context = spread(rng, 1, max(1, min(131072, room)))
        window = rng.choice((0, 0, 0, spread(rng, 1, 1000)))
        return dict(op=op, batch=batch, queries=queries, heads=heads, group=group, dim=dim, page=page, type=kind,
                    cache=cache, context=context, ragged=rng.random() < 0.7, window=window, shape=shape)
    heads, group = spread(rng, 1, 8), spread(rng, 1, 16)
    past = rng.choice((0, 0, spread(rng, 1, 4096)))
    most = spread(rng, 1, 16384)
    batch = 1 if most == 1 else spread(rng, 1, min(32, most))
    while heads * group * most * (most / 2 + past) * dim > 32 * 16384 * 8192 * 128:   # at most the largest listed case's work
        most = max(1, most * 3 // 4)
        batch = min(batch, most)
    return dict(op=op, batch=batch, most=most, past=past, heads=heads, group=group, dim=dim, type=kind,
                window=rng.choice((0, 0, 0, spread(rng, 1, 2000))), ragged=batch > 1, shape=shape)


def parts(case):
    """The tokens that each request of a packed batch brings: `most` in all, one at least where they suffice."""
    n, total = case["batch"], case["most"]
    if not case["ragged"]:
        return [total] * n
    rng = random.Random(case["shape"])
    cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def pasts(case):
    """The positions that each request of a packed batch has already."""
    rng = random.Random(case["shape"] + 1)
    most = case["past"] if case["op"] == "prompt" else case["context"]
    if case["op"] == "prompt" and not most:
        return [0] * case["batch"]
    return [rng.randrange(most + 1) for _ in range(case["batch"])]


def visible(case):
    """Visible lengths [request][query] of a decode case: the newest query sees the whole context."""
    rng = random.Random(case["shape"])
    ends = [rng.randint(max(1, case["context"] // 50), case["context"]) if case["ragged"] else case["context"]
            for _ in range(case["batch"])]
    return [[max(0, e - case["queries"] + 1 + i) for i in range(case["queries"])] for e in ends]


def work(case):
    op, dim, heads = case["op"], case["dim"], case["heads"]
    if op == "write":
        tokens = sum(parts(case))
        return {"bytes": 2 * tokens * heads * dim * (2 + SIZE[case["cache"]]), "flops": 0}
    low = (lambda e: max(0, e - case["window"])) if case["window"] else (lambda e: 0)
    if op == "decode":
        vis = visible(case)
        held = sum(max(r) - low(min(r)) for r in vis)
        seen = sum(e - low(e) for r in vis for e in r)
        rows = case["batch"] * case["queries"] * heads * case["group"]
        return {"bytes": 2 * held * heads * dim * SIZE[case["cache"]] + 2 * rows * dim * 2 + rows * 4,
                "flops": 4 * seen * heads * case["group"] * dim}
    seen, tokens, keys = 0, 0, 0
    for n, past in zip(parts(case), pasts(case)):
        w = case["window"] or n + past
        whole = max(0, min(n, w - past))                      # queries that still see everything before them
        seen += whole * past + whole * (whole + 1) // 2 + (n - whole) * w
        tokens, keys = tokens + n, keys + (n and min(n + past, n + w - 1))
    q = heads * case["group"] * dim
    return {"bytes": 2 * (2 * tokens * q + 2 * keys * heads * dim) + 4 * tokens * heads * case["group"],
            "flops": 4 * seen * q}


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
    kind = TYPES[case["cache"]]
    pools = []
    for _ in range(2):
        pool = torch.empty(total, heads, page, dim, dtype=kind, device="cuda")
        for lo in range(0, total, 4096):
            part = pool[lo:lo + 4096]
            part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
        pools.append(pool)
    return pools[0], pools[1], table


def starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dim, heads, kind = case["dim"], case["heads"], TYPES[case["type"]]

    def normal(*shape, by=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * by).to(kind)

    s = dict(case=case)
    if case["op"] == "write":
        new, past = parts(case), pasts(case)
        s["k_pages"], s["v_pages"], s["table"] = pages_of(case, [a + b for a, b in zip(new, past)], g)
        # keys and values as one projection leaves them: interleaved rows of one buffer
        both = normal(sum(new), 2, heads, dim)
        s["k"], s["v"] = both[:, 0], both[:, 1]
        s["cu"], s["start"] = starts(new), torch.tensor(past, dtype=torch.int64, device="cuda")
        s["k_scale"], s["v_scale"] = (0.03125, 0.0234375) if case["cache"] == "e4m3" else (1.0, 1.0)
    elif case["op"] == "decode":
        vis = visible(case)
        s["longest"] = max(max(r) for r in vis)
        s["k_pages"], s["v_pages"], s["table"] = pages_of(case, [max(r) for r in vis], g)
        s["vis"] = torch.tensor(vis, dtype=torch.int32, device="cuda")
        s["q"] = normal(case["batch"], case["queries"], heads * case["group"], dim, by=2.0)
        s["k_scale"], s["v_scale"] = (0.75, 1.25) if case["cache"] == "e4m3" else (1.0, 1.0)
    else:
        new, past = parts(case), pasts(case)
        s["cu_q"] = starts(new)
        s["cu_k"] = starts([a + b for a, b in zip(new, past)])
        s["q"] = normal(sum(new), heads * case["group"], dim, by=2.0)
        both = normal(sum(new) + sum(past), 2, heads, dim)
        s["k"], s["v"] = both[:, 0], both[:, 1]
    if case["op"] != "write":
        s["scale"] = 1.0 / math.sqrt(dim)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:-1], dtype=torch.float32, device="cuda")
    if own:
        import hierarchical_sparse_attention_index_gb300 as H
        if case["op"] != "prompt":
            s["cache"] = H.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["k_scale"], s["v_scale"])
        if case["op"] == "decode":
            s["ws"] = H.new_paged_workspace(s["cache"], heads * case["group"], case["queries"], s["longest"])
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        import hierarchical_sparse_attention_index_gb300 as H
        if case["op"] == "write":
            H.hsa_paged_cache_write(s["cache"], s["k"], s["v"], cu=s["cu"], start=s["start"])
            return s["k_pages"], s["v_pages"]
        if case["op"] == "decode":
            H.hsa_paged_attn_decode(s["cache"], s["q"], s["vis"], s["longest"], s["scale"], s["out"], s["ws"],
                                    window=case["window"], lse=s["lse"])
        else:
            H.hsa_prompt_attn(s["q"], s["k"], s["v"], s["cu_q"], s["scale"], s["out"], cu_k=s["cu_k"],
                              window=case["window"], lse=s["lse"])
        return s["out"], s["lse"]
    if case["op"] == "write":
        return plain_write(s)
    return plain_decode(s) if case["op"] == "decode" else plain_prompt(s)


def plain_write(s):
    case = s["case"]
    cu, page = s["cu"].long(), case["page"]
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    at = s["start"][b] + t - cu[b]
    where = s["table"][b, at // page].long()
    for pool, rows, scale in ((s["k_pages"], s["k"], s["k_scale"]), (s["v_pages"], s["v"], s["v_scale"])):
        if case["cache"] == "e4m3":
            rows = (rows.float() / scale).clamp(-448, 448).to(pool.dtype)
            pool.view(torch.uint8)[where, :, at % page] = rows.view(torch.uint8)
        else:
            pool[where, :, at % page] = rows
    return s["k_pages"], s["v_pages"]


def plain_decode(s):
    case = s["case"]
    batch, heads, dim, page, nq = case["batch"], case["heads"], case["dim"], case["page"], case["queries"]
    where = s["table"].clamp(min=0).long()
    k, v = (p.view(torch.uint8)[where].view(p.dtype) if p.dtype == TYPES["e4m3"] else p[where]
            for p in (s["k_pages"], s["v_pages"]))
    k, v = (x.float().transpose(2, 3).reshape(batch, -1, heads, dim) for x in (k, v))   # [b][position][head][dim]
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


def plain_prompt(s):
    case = s["case"]
    heads, group, dim = case["heads"], case["group"], case["dim"]
    new, past = parts(case), pasts(case)
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    q0 = k0 = 0
    for n, old in zip(new, past):
        k, v = (x[k0:k0 + n + old].float() for x in (s["k"], s["v"]))
        for lo in range(0, n, 2048):                # blocks of queries, so that the weights of long prompts fit
            hi = min(n, lo + 2048)
            first = max(0, lo + old + 1 - case["window"]) if case["window"] else 0
            q = s["q"][q0 + lo:q0 + hi].float().view(hi - lo, heads, group, dim)
            ends = torch.arange(lo, hi, device="cuda")[:, None] + old
            at = torch.arange(first, hi + old, device="cuda")
            seen = at <= ends
            if case["window"]:
                seen &= at > ends - case["window"]
            x = torch.einsum("ihgd,thd->hgit", q, k[first:hi + old]) * s["scale"]
            x = x.masked_fill(~seen, -math.inf)
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            total = p.sum(-1, keepdim=True)
            o = torch.einsum("hgit,thd->ihgd", p / total, v[first:hi + old])
            out[q0 + lo:q0 + hi] = o.reshape(hi - lo, heads * group, dim)
            lse[q0 + lo:q0 + hi] = (torch.log(total) + top)[..., 0].permute(2, 0, 1).reshape(hi - lo, -1)
        q0, k0 = q0 + n, k0 + n + old
    return out, lse


# ------------------------------------------------------------------------- the definition, 64 bits
def to_e4m3(x):
    """The nearest E4M3 value of each element (ties to the even one), beyond 448 the border."""
    size = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(size.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(size / step) * step).clamp(max=448.0)


def exact(case, seed):
    s = prepare(case, seed)
    dim, heads = case["dim"], case["heads"]
    if case["op"] == "write":
        pools = [s["k_pages"].double(), s["v_pages"].double()]
        t0 = 0
        for b, (n, old) in enumerate(zip(parts(case), pasts(case))):
            at = 0
            while at < n:                           # page by page
                first = (old + at) % case["page"]
                take = min(n - at, case["page"] - first)
                where = int(s["table"][b, (old + at) // case["page"]])
                for pool, rows, scale in zip(pools, (s["k"], s["v"]), (s["k_scale"], s["v_scale"])):
                    x = rows[t0 + at:t0 + at + take].double() / scale
                    pool[where, :, first:first + take] = (to_e4m3(x) if case["cache"] == "e4m3" else x).transpose(0, 1)
                at += take
            t0 += n
        return tuple(pools)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")

    def attend(q, k, v, ends, w):
        """q [n][group][dim], k and v [t][dim], ends [n]: query i weighs the keys max(0, ends[i] - w) .. ends[i] - 1."""
        x = (q.reshape(-1, dim) @ k.T).view(q.shape[0], -1, k.shape[0]) * s["scale"]
        at = torch.arange(k.shape[0], device="cuda")[None, :]
        hide = (at >= ends[:, None]) | (at < ends[:, None] - w)
        x.masked_fill_(hide[:, None, :], -math.inf)
        l = torch.logsumexp(x, -1)
        x.sub_(l[..., None]).exp_()
        x.nan_to_num_(nan=0.0)                      # a query that sees no key has the output 0
        return (x.view(-1, k.shape[0]) @ v).view(q.shape), l

    group, w = case["group"], case["window"] or 1 << 40
    if case["op"] == "decode":
        for b, ends in enumerate(visible(case)):
            n = max(ends)
            if not n:
                continue
            where = s["table"][b, :-(-n // case["page"])].long()
            at = torch.tensor(ends, device="cuda")
            for h in range(heads):
                k, v = (p.view(torch.uint8)[where, h].view(p.dtype) if p.element_size() == 1 else p[where, h]
                        for p in (s["k_pages"], s["v_pages"]))
                o, l = attend(s["q"][b, :, h * group:(h + 1) * group].double(),
                              k.double().reshape(-1, dim)[:n] * s["k_scale"], v.double().reshape(-1, dim)[:n] * s["v_scale"],
                              at, w)
                out[b, :, h * group:(h + 1) * group], lse[b, :, h * group:(h + 1) * group] = o, l
        return out, lse
    q0 = k0 = 0
    for n, old in zip(parts(case), pasts(case)):
        for h in range(heads):
            mine = slice(h * group, (h + 1) * group)
            for lo in range(0, n, 1024):
                hi = min(n, lo + 1024)
                first = max(0, lo + old + 1 - w)
                ends = torch.arange(lo, hi, device="cuda") + old + 1 - first
                k, v = (x[k0 + first:k0 + old + hi, h].double() for x in (s["k"], s["v"]))
                o, l = attend(s["q"][q0 + lo:q0 + hi, mine].double(), k, v, ends, w)
                out[q0 + lo:q0 + hi, mine], lse[q0 + lo:q0 + hi, mine] = o, l
        q0, k0 = q0 + n, k0 + n + old
    return out, lse
