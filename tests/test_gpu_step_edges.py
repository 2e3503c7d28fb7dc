"""Edges of the calls of a speculative step: waits that run out, long tails of small weights, places in the batch, many requests,
results off 32-byte boundaries, rows far apart, and steps with more query rows than the warp kernel takes. Bounds: tests/dense.py
and tests/test_gpu_step.py."""
import pytest
import torch

from tests import dense as D
from tests import four
from tests import test_gpu_dense_edges as E
from tests import test_gpu_step as S
from tests.test_gpu_step import BF, F4, F8, HF, H, check_decode, clean, i32, starts  # noqa: F401  (H is a fixture)

pytestmark = pytest.mark.gpu


def test_waits_that_run_out(H):  # noqa: F811
    """With a wait limit of 1 ns the kernel for many rows gives up over 4-bit pages, too: it ends by itself, the flag is set, the
    next call is not affected."""
    cache = S.cache_of(H, [65536], 1, 128, 64, F4, 3)
    cache = H.PagedCache(cache.k, cache.v, cache.table.expand(200, -1).contiguous(), 1.0, 1.0, cache.k_s, cache.v_s)
    q = torch.randn(200, 5, 8, 128, generator=torch.Generator().manual_seed(9)).to(BF).cuda()          # 40 rows per key head
    vis = torch.full((200, 5), 65536, dtype=torch.int32).cuda()
    ws = H.new_paged_workspace(cache, 8, 5, 65536)

    def call():
        out = torch.zeros_like(q)
        H.hsa_paged_attn_decode(cache, q, vis, 65536, 0.1, out, ws)
        return out, H.hsa_get_device_status()

    want = call()
    assert want[1] == (0, 0)
    try:
        H.hsa_set_wait_limit(1)
        short = call()
    finally:
        H.hsa_set_wait_limit(0)
    assert short[1] == (H.STATUS_CODES["HSA_ERR_TIMEOUT"], H.HSA_FLAG_TIMEOUT)
    again = call()
    assert again[1] == (0, 0) and torch.equal(again[0], want[0])


@pytest.mark.parametrize("gap", [14.0, 16.0, 17.4])
@pytest.mark.parametrize("qt", [BF, HF])
@pytest.mark.parametrize("dim,group", [(128, 8), (64, 16), (128, 28), (64, 64)])
def test_decode_long_tail(H, qt, dim, group, gap):  # noqa: F811
    """A few keys far above 65,529 alike: the tail's weights are 2^-20 and less, and what they bring together is kept."""
    n, heads, page, batch = 65536, 4, 64, 128
    at = [0, 16, 32, 48, n // 4, n // 2, 3 * n // 4]
    q, k, v = E.tail(n, heads, dim, torch.float32, at, gap)
    pages = n // page
    pools = []
    for x, keys in ((k, True), (v, False)):
        pools.append(four.pack(x.view(pages, page, heads, dim).transpose(1, 2).contiguous().cuda(), keys))
    (k, ks), (v, vs) = pools
    table = torch.arange(pages, dtype=torch.int32).cuda().repeat(batch, 1)
    q = q.to(qt).cuda().expand(batch, 1, heads * group, dim).contiguous()
    cache = H.PagedCache(k, v, table, 1.0, 1.0, ks, vs)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    vis = torch.full((batch, 1), n, dtype=torch.int32, device="cuda")
    scale = dim ** -0.5
    H.hsa_paged_attn_decode(cache, q, vis, n, scale, out, H.new_paged_workspace(cache, heads * group, 1, n), lse=lse)
    clean(H)
    kk, vv = D.unpage(four.unpack(k, ks, True), table, 0, n)[0], D.unpage(four.unpack(v, vs, False), table, 0, n)[0]
    hi = torch.full((1,), n, device="cuda")
    for h in range(heads):
        row = q[0, 0, h * group][None].double()
        o, l, A, mag = D.attention(row, kk[:, h], vv[:, h], hi * 0, hi, scale)
        A = E.with_floor(A, n, vv, HF, qt, l, (row @ kk[:, h].T).max() * scale)
        for r in (h * group, (h + 1) * group - 1):
            D.check(out[0, :1, r], lse[0, :1, r], o, l, A, mag, n, dim, HF, f"head {h}")
    assert torch.equal(out[0], out[-1]) and torch.equal(lse[0], lse[-1])


@pytest.mark.parametrize("group,nq", [(7, 5), (8, 1), (4, 3), (16, 8), (23, 1)])
def test_decode_does_not_depend_on_the_place_in_the_batch(H, group, nq):  # noqa: F811
    ends = [700, 33, 5, 1900, 0, 1024, 64, 2047]
    cache = S.cache_of(H, ends, 2, 128, 48, F4, 4)
    vis = i32([[max(0, e - nq + 1 + i) for i in range(nq)] for e in ends])
    q = torch.randn(8, nq, 2 * group, 128).to(BF).cuda()

    def call(order):
        c = H.PagedCache(cache.k, cache.v, cache.table[order].contiguous(), 1.0, 1.0, cache.k_s, cache.v_s)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        H.hsa_paged_attn_decode(c, q[order].contiguous(), vis[order].contiguous(), 2047, 0.1, out, H.new_paged_workspace(c, 2 * group, nq, 2047), lse=lse)
        clean(H)
        return out, lse

    order = torch.tensor([3, 1, 7, 0, 5, 4, 6, 2]).cuda()
    a, b = call(torch.arange(8).cuda()), call(order)
    assert torch.equal(a[0][order], b[0]) and torch.equal(a[1][order], b[1])
    again = call(order)
    assert torch.equal(again[0], b[0]) and torch.equal(again[1], b[1])


@pytest.mark.parametrize("nq,group", [(5, 7), (8, 16), (1, 8)])
@pytest.mark.parametrize("most", [900, 9000])
def test_decode_results_on_16_byte_boundaries(H, nq, group, most):  # noqa: F811
    """Outputs and workspaces that do not start on 32-byte boundaries give the same bits, and nothing around them changes."""
    cache = S.cache_of(H, [most, 300], 2, 128, 32, F4, 5)
    q = torch.randn(2, nq, 2 * group, 128).to(BF).cuda()
    vis = i32([[most - nq + 1 + i for i in range(nq)], [300 - nq + 1 + i for i in range(nq)]])
    ws = H.new_paged_workspace(cache, 2 * group, nq, most)
    want = torch.empty_like(q)
    H.hsa_paged_attn_decode(cache, q, vis, most, 0.1, want, ws)
    n = ws.numel()
    room, ws_room = torch.full((q.numel() + 16,), 7.0, dtype=BF, device="cuda"), torch.full((n + 64,), 9, dtype=torch.uint8, device="cuda")
    out = room[8:8 + q.numel()].view_as(q)
    H.hsa_paged_attn_decode(cache, q, vis, most, 0.1, out, ws_room[16:16 + n])
    clean(H)
    assert torch.equal(out, want)
    assert (room[:8] == 7).all() and (room[8 + q.numel():] == 7).all()
    assert (ws_room[:16] == 9).all() and (ws_room[16 + n:] == 9).all()


@pytest.mark.parametrize("kv", [BF, F8, F4])
def test_append_and_read_many_requests(H, kv):  # noqa: F811
    """More requests than cu in shared memory holds, most of them with a token or none."""
    batch, page, heads, dim = 1500, 16, 2, 64
    counts = [(7 * b) % 3 for b in range(batch)]
    past = [(5 * b) % 40 for b in range(batch)]
    S.append(H, counts, past, heads, 2, dim, page, BF, kv, 64, 0, True, scales=(0.5, 0.25) if kv in (F8, F4) else (1.0, 1.0), pad=5)
    cache = S.cache_of(H, [43] * batch, heads, dim, page, kv, 1)
    n = sum(counts)
    k, v = (torch.full((n + 3, heads, dim), 7.0, dtype=BF, device="cuda") for _ in range(2))
    H.hsa_paged_cache_read(cache, k, v, cu=starts(counts), start=torch.tensor(past).cuda())
    clean(H)
    b = torch.repeat_interleave(torch.arange(batch), torch.tensor(counts)).cuda()
    pos = torch.arange(n).cuda() - starts(counts)[b].long() + torch.tensor(past).cuda()[b]
    where = cache.table[b, pos // page].long()
    raw = torch.uint8 if kv in (F8, F4) else kv
    got = cache.k.view(raw)[where, :, pos % page]
    want = four.unpack(got, cache.k_s[where, :, pos % page], True) if kv == F4 else got.view(kv).double()
    assert torch.equal(k[:n].double(), want.to(BF).double()) and (k[n:] == 7).all() and (v[n:] == 7).all()


@pytest.mark.parametrize("kv", [BF, F4])
def test_rows_far_apart(H, kv):  # noqa: F811
    """Rows 2^27 elements apart, so that offsets pass 32 bits."""
    n, heads, dim, stride = 20, 1, 64, 1 << 27
    room = torch.zeros((n - 1) * stride + 4 * dim, dtype=BF, device="cuda")
    rows = [room[i * dim:].as_strided((n, heads, dim), (stride, dim, 1)) for i in range(4)]
    x = torch.randn(3, n, heads, dim).to(BF).cuda()
    for r, y in zip(rows, x):
        r.copy_(y)
    inv = torch.rand(32).cuda()
    caches = [S.cache_of(H, [n], heads, dim, 16, kv, 0) for _ in range(2)]
    close = torch.empty(n, heads, dim, dtype=BF, device="cuda")
    H.hsa_paged_cache_append(caches[0], rows[1], rows[2], inv, q=rows[0], q_out=rows[3])
    H.hsa_paged_cache_append(caches[1], x[1], x[2], inv, q=x[0], q_out=close)
    assert torch.equal(rows[3], close)
    for a, b in zip(S.copies(caches[0]), S.copies(caches[1])):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    k, v = torch.empty_like(close), torch.empty_like(close)
    H.hsa_paged_cache_read(caches[0], rows[0], rows[1])
    H.hsa_paged_cache_read(caches[1], k, v)
    clean(H)
    assert torch.equal(rows[0], k) and torch.equal(rows[1], v)


def test_append_with_more_heads_than_a_block_takes(H):  # noqa: F811
    """One token with 1,024 key heads and 4,096 query heads."""
    S.append(H, [1], [3], 1024, 4, 64, 16, BF, F4, 64, 0, True, scales=(0.5, 0.25))
    S.append(H, [2, 1], [0, 30], 300, 3, 128, 16, HF, HF, 96, 32, False)


@pytest.mark.parametrize("group", [5, 10, 30])
def test_steps_captured_and_at_the_same_time(H, group):  # noqa: F811
    """Whole steps with 20, 40 and 120 query rows: three replays of a graph, and steps on three streams at once, give the bits of
    steps one by one."""
    want = []
    for seed in range(3):
        s = S.new_step(H, seed, group=group)
        for _ in range(3):
            S.step(H, s)
        want.append([s[x].clone() for x in S.KEYS])
    states = [S.new_step(H, seed, group=group) for seed in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(3):
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                S.step(H, s)
    torch.cuda.synchronize()
    for s, w in zip(states, want):
        assert all(torch.equal(s[x], y) for x, y in zip(S.KEYS, w))
    s = S.new_step(H, 0, group=group)
    first, pages = s["start"].clone(), S.copies(s["cache"])
    with torch.cuda.stream(torch.cuda.Stream()):
        S.step(H, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        S.step(H, s)
    s["start"].copy_(first)
    for t, old in zip((s["cache"].k, s["cache"].v, s["cache"].k_s, s["cache"].v_s), pages):
        t.copy_(old)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s[x], y) for x, y in zip(S.KEYS, want[0]))
    clean(H)


def test_two_graphs_that_share_a_workspace(H):  # noqa: F811
    """Graphs captured with one workspace and replayed in turn on one stream do not disturb each other."""
    a, b = (S.new_step(H, seed, batch=1, most=9000, group=group) for seed, group in ((1, 2), (2, 10)))
    big = max(a["ws"].numel(), b["ws"].numel())
    shared = torch.empty(big, dtype=torch.uint8, device="cuda")
    outs = []
    for s in (a, b):
        s["start"].fill_(8000)
        s["vis"].copy_(8000 + s["ahead"])
        q = s["q"].reshape(s["out"].shape).contiguous()
        s["fixed"] = q
        H.hsa_paged_attn_decode(s["cache"], q, s["vis"], s["most"], s["scale"], s["out"], s["ws"])
        outs.append(s["out"].clone())
    torch.cuda.synchronize()
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            H.hsa_paged_attn_decode(s["cache"], s["fixed"], s["vis"], s["most"], s["scale"], s["out"], shared)
        graphs.append(g)
    for _ in range(3):
        for s in (a, b):
            s["out"].zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a["out"], outs[0]) and torch.equal(b["out"], outs[1])
    clean(H)


def test_verify_of_garbage_stays_in_range(H):  # noqa: F811
    """Rows that are no distributions (too large a sum, random bits): tokens stay inside the vocabulary, nothing else is written."""
    batch, nq, n = 40, 4, 5003
    g = torch.Generator().manual_seed(1)
    for p in (torch.ones(batch, nq, n), torch.randint(-2 ** 31, 2 ** 31 - 1, (batch, nq, n), generator=g, dtype=torch.int32).view(torch.float32)):
        p = p.cuda()
        q = p[:, 1:].contiguous().flip(1)
        drafted = torch.randint(0, n, (batch, nq - 1), generator=g, dtype=torch.int32).cuda()
        room = torch.full((batch * nq + 32,), 55, dtype=torch.int32, device="cuda")
        tokens, accepted = room[16:16 + batch * nq].view(batch, nq), torch.full((batch,), 55, dtype=torch.int32, device="cuda")
        H.hsa_draft_verify(p, q, drafted, torch.rand(batch, nq - 1).cuda(), torch.rand(batch).cuda(), accepted, tokens)
        code, _ = H.hsa_get_device_status()
        assert code == 0 and ((accepted >= 0) & (accepted < nq)).all()
        assert ((tokens >= -1) & (tokens < n)).all() and (room[:16] == 55).all() and (room[16 + batch * nq:] == 55).all()


def test_calls_refuse_other_devices_and_types(H):  # noqa: F811
    cache = S.cache_of(H, [64], 2, 64, 16, F4, 0)
    x = torch.randn(4, 2, 64).to(BF).cuda()
    inv = torch.ones(32).cuda()
    for bad in (dict(k=x.cpu()), dict(v=x.half()), dict(inv_freq=inv.cpu()), dict(inv_freq=inv.double()), dict(q=x), dict(q=x, q_out=x[:2]),
                dict(q=x, q_out=x.half()), dict(cu=i32([0, 4]).long()), dict(start=i32([0])), dict(q=x.cpu(), q_out=x)):
        with pytest.raises(ValueError):
            H.hsa_paged_cache_append(cache, **{**dict(k=x, v=x, inv_freq=inv), **bad})
    for bad in (dict(k=x.cpu()), dict(v=x.half()), dict(cu=i32([0]))):
        with pytest.raises(ValueError):
            H.hsa_paged_cache_read(cache, **{**dict(k=x.clone(), v=x.clone()), **bad})
    ok = dict(p=torch.rand(2, 3, 50).cuda(), q=torch.rand(2, 2, 50).cuda(), drafted=i32([[1, 2], [3, 4]]), u_accept=torch.rand(2, 2).cuda(),
              u_sample=torch.rand(2).cuda(), accepted=i32([0, 0]), tokens=i32([[0] * 3] * 2))
    for bad in (dict(p=ok["p"].cpu()), dict(p=ok["p"].double()), dict(q=ok["q"].half()), dict(q=ok["p"]), dict(drafted=ok["drafted"].long()),
                dict(u_sample=ok["u_sample"].double()), dict(tokens=ok["drafted"]), dict(n_draft=i32([1]))):
        with pytest.raises(ValueError):
            H.hsa_draft_verify(**{**ok, **bad})
    clean(H)


@pytest.mark.parametrize("dtype", [torch.float32, BF, HF])
@pytest.mark.parametrize("n,lookup", [(131072, False), (131071, False), (32000, False), (131072, True), (2047, False)])
def test_verify_does_not_depend_on_the_batch(H, dtype, n, lookup):  # noqa: F811
    """The same requests among 6 to 300 others, which take other numbers and sizes of CTAs: the same tokens."""
    g = torch.Generator().manual_seed(n)
    few, nq = 3, 2
    p, q = (torch.softmax(3 * torch.randn(few, r, n, generator=g), -1).to(dtype).cuda() for r in (nq, nq - 1))
    drafted = torch.randint(0, n, (few, nq - 1), generator=g, dtype=torch.int32).cuda()
    u, v = torch.tensor([[0.0], [2.0], [0.5]]).cuda(), torch.rand(few, generator=g).cuda()
    want = None
    for times in (2, 7, 11, 34, 100):
        batch = few * times
        tokens, accepted = torch.full((batch, nq), 55, dtype=torch.int32, device="cuda"), torch.full((batch,), 55, dtype=torch.int32, device="cuda")
        H.hsa_draft_verify(p.repeat(times, 1, 1), None if lookup else q.repeat(times, 1, 1), drafted.repeat(times, 1), u.repeat(times, 1),
                           v.repeat(times), accepted, tokens)
        clean(H)
        want = want or (accepted[:few], tokens[:few])
        for got, w in zip((accepted, tokens), want):
            assert torch.equal(got.view(times, few, *got.shape[1:]), w.expand(times, *w.shape))
