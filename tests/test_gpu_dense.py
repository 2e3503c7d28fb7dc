"""Dense attention calls on the GPU against plain 64-bit forms (bounds: tests/dense.py): paged cache
writes, paged decode attention and packed prompt attention, at the sizes, masks, strides and types
where they can go wrong, and together as a layer uses them."""
import math

import pytest
import torch

from tests import dense as D

pytestmark = pytest.mark.gpu

BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def H():
    import hierarchical_sparse_attention_index_gb300 as h
    h.load_library()
    return h


def clean(H, want=0):
    code, flags = H.hsa_get_device_status()
    assert flags == want and code == 0, (code, flags)


def decode(H, batch, nq, heads, group, dim, page, kv, qt, vis, window=0, max_vis=None, seed=0, poison=True, scales=(1., 1.),
           q_by=2.0, table_edit=None, flags=0, lse=True):
    """Run a decode call and compare every row with the 64-bit form; returns the output."""
    longest = [max(r) for r in vis]
    k, v, table = D.paged(batch, longest, heads, dim, page, kv, seed)
    if poison:      # what no query sees may hold anything
        seen = torch.zeros(k.shape[0], page, dtype=torch.bool)
        for b, r in enumerate(vis):
            low = min([max(0, x - window) if window else 0 for x in r if x > 0], default=0)
            for t in range(low, longest[b]):
                seen[table[b, t // page].long(), t % page] = True
        bad = torch.tensor([math.nan, math.inf, -math.inf]).to(kv) if kv != F8 else torch.tensor([math.nan] * 3).to(kv)
        raw = torch.uint8 if kv == F8 else torch.int16
        fill = bad.view(raw)[torch.randint(0, 3, k.shape)]
        for x in (k, v):
            x.view(raw).copy_(torch.where(seen[:, None, :, None], x.view(raw), fill))
    if table_edit:
        table_edit(table)
    if max_vis is not None:                     # the table's rows reach max_vis; no position needs their ends
        table = torch.cat([table, table.new_full((batch, -(-max_vis // page)), -1)], 1)
    k, v, table = k.cuda(), v.cuda(), table.cuda()
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(batch, nq, heads * group, dim, generator=g) * q_by).to(qt).cuda()
    vis_d = torch.tensor(vis, dtype=torch.int32).cuda()
    cache = H.PagedCache(k, v, table, *scales)
    max_vis = max(longest) if max_vis is None else max_vis
    out = torch.full_like(q, 7.0)
    l_out = torch.full(q.shape[:3], 7.0, device="cuda") if lse else None
    ws = H.new_paged_workspace(cache, heads * group, nq, max_vis)
    ws.fill_(0xFF)                              # the workspace needs no initialisation
    scale = 1 / math.sqrt(dim)
    H.hsa_paged_attn_decode(cache, q, vis_d, max_vis, scale, out, ws, window=window, lse=l_out)
    clean(H, flags)
    p_type = BF if kv == BF else HF
    for b in range(batch):
        n = longest[b]
        kk, ok = D.unpage(k, table, b, n)
        vv, _ = D.unpage(v, table, b, n)
        hi = torch.tensor(vis[b], device="cuda").repeat_interleave(group)
        lo = (hi - window).clamp(min=0) if window else torch.zeros_like(hi)
        for h in range(heads):
            rows = q[b, :, h * group:(h + 1) * group].reshape(-1, dim).double()
            kh, vh = kk[:, h] * scales[0], vv[:, h] * scales[1]
            kh, vh = kh.nan_to_num(0, 0, 0) if poison else kh, vh.nan_to_num(0, 0, 0) if poison else vh
            o, l, A, mag = D.attention(rows, kh, vh, lo, hi, scale, ok)
            got = out[b, :, h * group:(h + 1) * group].reshape(-1, dim)
            got_l = l_out[b, :, h * group:(h + 1) * group].reshape(-1) if lse else None
            D.check(got, got_l, o, l, A, mag, n, dim, p_type, f"request {b} head {h}")
    return out


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv,qt", [(BF, BF), (HF, HF), (F8, BF), (F8, HF)])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 255, 256, 257, 1000])
def test_decode_lengths(H, dim, kv, qt, n):
    decode(H, 1, 1, 2, 4, dim, 16, kv, qt, [[n]], seed=n, scales=(0.5, 1.5) if kv == F8 else (1., 1.))


@pytest.mark.parametrize("kv,qt", [(BF, BF), (HF, HF), (F8, BF)])
@pytest.mark.parametrize("dim,heads,group,nq,page", [
    (128, 1, 1, 1, 16), (128, 3, 7, 5, 48), (64, 5, 3, 8, 32), (128, 2, 16, 1, 64), (64, 1, 17, 1, 80), (128, 1, 32, 1, 16),
    (128, 1, 33, 1, 128), (64, 2, 16, 4, 64), (128, 1, 128, 8, 256), (64, 16, 1, 3, 16)])
def test_decode_layouts(H, kv, qt, dim, heads, group, nq, page):
    batch = 3
    ends = [700, 33, 5]
    vis = [[max(0, e - nq + 1 + i) for i in range(nq)] for e in ends[:batch]]
    decode(H, batch, nq, heads, group, dim, page, kv, qt, vis, seed=group * nq)


@pytest.mark.parametrize("kv", [BF, F8])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 128, 5000])
def test_decode_window(H, kv, window):
    """A sliding window; queries one apart, and queries far apart (more keys than the window's splits assume)."""
    decode(H, 2, 3, 2, 4, 128, 32, kv, BF, [[998, 999, 1000], [4, 5, 6]], window=window)
    decode(H, 1, 3, 1, 2, 64, 16, kv, BF, [[40, 2000, 900]], window=window)


@pytest.mark.parametrize("kv", [BF, HF])
@pytest.mark.parametrize("dim,group,nq,page", [(128, 5, 5, 16), (64, 25, 1, 48), (128, 26, 1, 32), (64, 7, 5, 64), (128, 16, 8, 128),
                                               (128, 128, 1, 80), (64, 127, 2, 16), (128, 1, 8, 16)])
def test_decode_more_work_than_places(H, kv, dim, group, nq, page):
    """Ragged batches with more pieces of work than the GPU holds at a time, empty requests among them; queries of one
    request need not stand one behind the other."""
    batch = 90
    vis = [[(37 * b * b + 11 * i) % 500 if b % 7 else 0 for i in range(nq)] for b in range(batch)]
    decode(H, batch, nq, 2, group, dim, page, kv, kv, vis, seed=group, max_vis=520)


@pytest.mark.parametrize("kv,group,nq", [(BF, 5, 5), (HF, 8, 1), (F8, 8, 1), (BF, 1, 1)])
@pytest.mark.parametrize("dim", [64, 128])
def test_decode_many_splits(H, kv, group, nq, dim):
    """One request and key head with more splits than one warp joins."""
    decode(H, 1, nq, 1, group, dim, 64, kv, BF if kv == F8 else kv, [[20001 + i for i in range(nq)]], seed=nq, scales=(0.5, 1.5) if kv == F8 else (1., 1.))


def test_decode_results_on_16_byte_boundaries(H):
    """Outputs and workspaces that do not start on 32-byte boundaries give the same bits, and nothing around them changes."""
    k, v, table = D.paged(2, [900, 300], 2, 128, 32, BF, 5)
    cache = H.PagedCache(k.cuda(), v.cuda(), table.cuda())
    for nq, group in ((5, 7), (1, 4)):
        q = torch.randn(2, nq, 2 * group, 128).to(BF).cuda()
        vis = torch.tensor([[896 + i for i in range(nq)], [296 + i for i in range(nq)]], dtype=torch.int32).cuda()
        ws = H.new_paged_workspace(cache, 2 * group, nq, 900)
        want = torch.empty_like(q)
        H.hsa_paged_attn_decode(cache, q, vis, 900, 0.1, want, ws)
        n = ws.numel()
        room, ws_room = torch.full((q.numel() + 16,), 7.0, dtype=BF, device="cuda"), torch.full((n + 64,), 9, dtype=torch.uint8, device="cuda")
        out = room[8:8 + q.numel()].view_as(q)
        H.hsa_paged_attn_decode(cache, q, vis, 900, 0.1, out, ws_room[16:16 + n])
        clean(H)
        assert torch.equal(out, want)
        assert (room[:8] == 7).all() and (room[8 + q.numel():] == 7).all()
        assert (ws_room[:16] == 9).all() and (ws_room[16 + n:] == 9).all()


def test_decode_empty_requests(H):
    """Requests and queries with nothing visible: output 0, lse -inf, also beside long ones."""
    decode(H, 4, 2, 2, 3, 128, 16, BF, BF, [[0, 0], [0, 1], [0, 900], [5, 0]], max_vis=1000)
    out = decode(H, 2, 1, 1, 1, 64, 16, HF, HF, [[0], [0]], max_vis=16)
    assert (out == 0).all()


@pytest.mark.parametrize("max_vis", [700, 5000, 60000])
def test_decode_bound_above_the_lengths(H, max_vis):
    """max_vis is only an upper bound: the same rows whatever it is (within the bounds)."""
    longest = 700
    k, v, table = D.paged(2, [longest, 64], 2, 128, 32, BF, 3)
    wide = torch.full((2, max(table.shape[1], -(-max_vis // 32))), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    g = torch.Generator().manual_seed(1)
    q = torch.randn(2, 1, 8, 128, generator=g).to(BF).cuda()
    cache = H.PagedCache(k.cuda(), v.cuda(), wide.cuda())
    ws = H.new_paged_workspace(cache, 8, 1, max_vis)
    out, lse = torch.empty_like(q), torch.empty(2, 1, 8, device="cuda")
    vis = torch.tensor([[longest], [64]], dtype=torch.int32).cuda()
    H.hsa_paged_attn_decode(cache, q, vis, max_vis, 0.1, out, ws, lse=lse)
    clean(H)
    for b, n in enumerate((longest, 64)):
        kk, ok = D.unpage(cache.k, cache.table, b, n)
        vv, _ = D.unpage(cache.v, cache.table, b, n)
        for h in range(2):
            hi = torch.full((4,), n, device="cuda")
            o, l, A, mag = D.attention(q[b, 0, 4 * h:4 * h + 4].double(), kk[:, h], vv[:, h], hi * 0, hi, 0.1)
            D.check(out[b, 0, 4 * h:4 * h + 4], lse[b, 0, 4 * h:4 * h + 4], o, l, A, mag, n, 128, BF)


def test_decode_large_and_small_values(H):
    """Logits up to thousands (one key takes all the weight), rising along the cache, and bf16 queries
    of any magnitude against an FP8 cache."""
    for by in (2.0 ** -30, 1.0, 60.0, 2.0 ** 12):
        decode(H, 1, 1, 2, 4, 128, 16, F8, BF, [[300]], q_by=by)
        decode(H, 1, 1, 2, 4, 64, 16, BF, BF, [[300]], q_by=by)
    dim, n = 128, 2000
    k, v, table = D.paged(1, [n], 1, dim, 16, HF, 5)
    rise = torch.linspace(0, 1, n)
    for t in range(n):      # logit of position t grows from 0 to about 90
        k[table[0, t // 16].long(), :, t % 16] = 0
        k[table[0, t // 16].long(), :, t % 16, 0] = rise[t] * 4
    q = torch.zeros(1, 1, 2, dim).to(HF)
    q[..., 0] = 256.0
    cache = H.PagedCache(k.cuda(), v.cuda(), table.cuda())
    out = torch.empty_like(q.cuda())
    lse = torch.empty(1, 1, 2, device="cuda")
    H.hsa_paged_attn_decode(cache, q.cuda(), torch.tensor([[n]], dtype=torch.int32).cuda(), n, 1 / math.sqrt(dim), out,
                            H.new_paged_workspace(cache, 2, 1, n), lse=lse)
    clean(H)
    kk, _ = D.unpage(cache.k, cache.table, 0, n)
    vv, _ = D.unpage(cache.v, cache.table, 0, n)
    hi = torch.full((2,), n, device="cuda")
    o, l, A, mag = D.attention(q[0, 0].double().cuda(), kk[:, 0], vv[:, 0], hi * 0, hi, 1 / math.sqrt(dim))
    D.check(out[0, 0], lse[0, 0], o, l, A, mag, n, dim, HF)


@pytest.mark.parametrize("window", [0, 1, 50, 500, 700, 792, 860, 934])
def test_decode_workspace_serves_every_window(H, window):
    """A window shortens the lengths that are split, which can make more splits; the workspace is asked for without it."""
    k, v, table = D.paged(1, [935], 4, 128, 32, BF, 21)
    cache = H.PagedCache(k.cuda(), v.cuda(), table.cuda())
    ws = H.new_paged_workspace(cache, 28, 5, 935)
    q = torch.randn(1, 5, 28, 128).to(BF).cuda()
    out = torch.empty_like(q)
    for longest in (935, 860, 400, 77):
        vis = torch.full((1, 5), longest, dtype=torch.int32).cuda()
        H.hsa_paged_attn_decode(cache, q, vis, longest, 0.1, out, ws, window=window)
        clean(H)
        ks, vs = (D.unpage(x.cuda(), table.cuda(), 0, longest)[0] for x in (k, v))
        lo = torch.full((35,), max(0, longest - window) if window else 0, device="cuda")
        hi = torch.full((35,), longest, device="cuda")
        for h in range(4):
            mine = slice(7 * h, 7 * h + 7)
            o, l, A, mag = D.attention(q[0, :, mine].reshape(-1, 128).double(), ks[:, h], vs[:, h], lo, hi, 0.1)
            D.check(out[0, :, mine].reshape(-1, 128), None, o, l, A, mag, longest, 128, BF, f"window {window} of {longest}")


def test_decode_bad_pages_and_lengths_are_flagged(H):
    """Page ids outside the pool are skipped, lengths outside [0, max_vis] cut; both set the flag."""
    def edit(table):
        table[0, 3] = -1
        table[0, 7] = 1 << 20
        table[1, 0] = -5
    decode(H, 2, 1, 2, 4, 128, 16, BF, BF, [[400], [16]], table_edit=edit, flags=H.HSA_FLAG_INDEX_RANGE, poison=False)
    k, v, table = D.paged(2, [64, 64], 1, 64, 16, BF, 3)
    cache = H.PagedCache(k.cuda(), v.cuda(), table.cuda())
    q = torch.randn(2, 1, 1, 64).to(BF).cuda()
    ws = H.new_paged_workspace(cache, 1, 1, 64)
    outs = []
    for vis in ([[64], [0]], [[1000], [-3]]):
        out = torch.empty_like(q)
        H.hsa_paged_attn_decode(cache, q, torch.tensor(vis, dtype=torch.int32).cuda(), 64, 0.1, out, ws)
        outs.append(out)
    clean(H, H.HSA_FLAG_INDEX_RANGE)
    assert torch.equal(outs[0], outs[1])


def test_decode_shared_pages_and_long_cache(H):
    """Requests that share prefix pages; and a pool past 2^31 bytes, read at its end."""
    n, dim, heads, page = 300, 128, 2, 16
    k, v, table = D.paged(1, [n], heads, dim, page, BF, 9)
    table = table.repeat(3, 1)
    q = torch.randn(1, 1, 4, dim).to(BF).repeat(3, 1, 1, 1).cuda()
    cache = H.PagedCache(k.cuda(), v.cuda(), table.cuda())
    out = torch.empty_like(q)
    H.hsa_paged_attn_decode(cache, q, torch.full((3, 1), n, dtype=torch.int32).cuda(), n, 0.1, out,
                            H.new_paged_workspace(cache, 4, 1, n))
    clean(H)
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
    big = (2 ** 31 + 2 ** 28) // (heads * 64 * dim * 2)
    kb = torch.zeros(big, heads, 64, dim, dtype=BF, device="cuda")
    vb = torch.zeros_like(kb)
    kb[-5:] = torch.randn(5, heads, 64, dim).to(BF).cuda()
    vb[-5:] = torch.randn(5, heads, 64, dim).to(BF).cuda()
    last = torch.arange(big - 5, big, dtype=torch.int32).cuda()[None]
    near = H.PagedCache(kb[-5:].contiguous(), vb[-5:].contiguous(), torch.arange(5, dtype=torch.int32).cuda()[None])
    far = H.PagedCache(kb, vb, last.contiguous())
    outs = []
    for c in (near, far):
        o = torch.empty_like(q[:1])
        H.hsa_paged_attn_decode(c, q[:1], torch.tensor([[311]], dtype=torch.int32).cuda(), 311, 0.1, o,
                                H.new_paged_workspace(c, 4, 1, 311))
        outs.append(o)
    clean(H)
    assert torch.equal(outs[0], outs[1])


# ------------------------------------------------------------------------------------- writes
def write_reference(pool, rows, table, cu, start, scale):
    pool = pool.clone()
    page, n_pages = pool.shape[2], pool.shape[0]
    f8 = pool.dtype == F8
    if f8:
        # the fp32 product with the scale's fp32 reciprocal
        inv = 1 / torch.tensor(scale, dtype=torch.float32)
        vals = (rows.float() * inv.to(rows.device)).clamp(-448, 448).to(F8).view(torch.uint8)
        nan = rows.isnan()
        vals = torch.where(nan, torch.tensor(0x7F, dtype=torch.uint8, device=rows.device), vals)
        target = pool.view(torch.uint8)
    else:
        vals, target = rows, pool
    skipped = False
    for b in range(table.shape[0]):
        for t in range(max(0, cu[b]), min(rows.shape[0], cu[b + 1])):
            pos = start[b] + t - cu[b]
            ok = 0 <= pos < table.shape[1] * page
            pg = int(table[b, pos // page]) if ok else -1
            if not ok or not 0 <= pg < n_pages:
                skipped = True
                continue
            target[pg, :, pos % page] = vals[t]
    return pool, skipped


@pytest.mark.parametrize("src,kv", [(BF, BF), (HF, HF), (BF, F8), (HF, F8)])
@pytest.mark.parametrize("heads,dim,page,counts,start", [
    (1, 64, 16, [1], [0]), (8, 128, 64, [1, 1, 1, 1], [5, 0, 63, 64]), (3, 64, 48, [0, 7, 0, 100, 1], [9, 0, 3, 47, 200]),
    (16, 128, 16, [33, 2], [15, 16]), (5, 128, 32, [0, 0, 65], [1, 2, 3]), (40, 128, 16, [3, 4], [1, 30])])
def test_write(H, src, kv, heads, dim, page, counts, start):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    pad = 3                                        # rows behind the last sequence
    k0, v0, table = D.paged(len(counts), [s + c for s, c in zip(start, counts)], heads, dim, page, kv, 4)
    both = torch.randn(cu[-1] + pad, 2, heads, dim) * 3
    both[0, 0, 0, :4] = torch.tensor([math.nan, math.inf, -math.inf, 60000.0])
    both = both.to(src).cuda()
    k, v = both[:, 0], both[:, 1]                   # rows 2 * heads * dim apart
    scales = (0.125, 0.3) if kv == F8 else (1., 1.)
    cache = H.PagedCache(k0.cuda(), v0.cuda(), table.cuda(), *scales)
    want = [write_reference(p, r, table, cu, start, s)[0] for p, r, s in ((cache.k, k, scales[0]), (cache.v, v, scales[1]))]
    H.hsa_paged_cache_write(cache, k, v, cu=torch.tensor(cu, dtype=torch.int32).cuda(),
                            start=torch.tensor(start, dtype=torch.int64).cuda())
    clean(H)
    raw = torch.uint8 if kv == F8 else torch.int16
    for got, ref in zip((cache.k, cache.v), want):
        a, b = got.view(raw), ref.view(raw)
        if kv == F8:                               # the sign of a NaN is not a value
            a, b = torch.where((a & 0x7F) == 0x7F, 0x7F, a), torch.where((b & 0x7F) == 0x7F, 0x7F, b)
        assert torch.equal(a, b)


def test_write_equal_shares_and_skips(H):
    """No cu: equal shares from position 0. Positions past the table or on bad pages are skipped and flagged."""
    k0, v0, table = D.paged(3, [40, 40, 40], 2, 64, 16, BF, 4)
    x = torch.randn(120, 2, 64).to(BF).cuda()
    cache = H.PagedCache(k0.cuda(), v0.cuda(), table.cuda())
    want, skipped = write_reference(cache.k, x, table, [0, 40, 80, 120], [0, 0, 0], 1.0)
    H.hsa_paged_cache_write(cache, x, x.clone())
    clean(H)
    assert not skipped and torch.equal(cache.k, want)
    table[1, 1], table[2, 0] = -1, 99
    cache = H.PagedCache(k0.cuda(), v0.cuda(), table.cuda())
    cu, start = [0, 50, 80, 120], [0, 0, -3]
    want, skipped = write_reference(cache.k, x, table, cu, start, 1.0)
    H.hsa_paged_cache_write(cache, x, x.clone(), cu=torch.tensor(cu, dtype=torch.int32).cuda(),
                            start=torch.tensor(start, dtype=torch.int64).cuda())
    clean(H, H.HSA_FLAG_WRITE_RANGE)
    assert skipped and torch.equal(cache.k, want)


def test_write_many_requests(H):
    """More requests than the search keeps in shared memory, some without rows."""
    batch, heads, dim, page = 1500, 1, 64, 16
    counts = [(7 * b) % 3 for b in range(batch)]
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    start = [b % 14 for b in range(batch)]
    k0, v0, table = D.paged(batch, [16] * batch, heads, dim, page, HF, 4)
    x = torch.randn(cu[-1], heads, dim).to(HF).cuda()
    cache = H.PagedCache(k0.cuda(), v0.cuda(), table.cuda())
    want, _ = write_reference(cache.k.cpu(), x.cpu(), table, cu, start, 1.0)
    H.hsa_paged_cache_write(cache, x, x, cu=torch.tensor(cu, dtype=torch.int32).cuda(),
                            start=torch.tensor(start, dtype=torch.int64).cuda())
    clean(H)
    assert torch.equal(cache.k.cpu(), want)


# ------------------------------------------------------------------------------------- prompts
def prompt(H, lens, heads, group, dim, dtype, past=None, window=0, seed=0, pad=0, strided=True, lse=True, cu_k=True, q_by=2.0):
    past = past or [0] * len(lens)
    cu_q, cu_kk = [pad], [pad]
    for n, o in zip(lens, past):
        cu_q.append(cu_q[-1] + n)
        cu_kk.append(cu_kk[-1] + max(0, n + o))
    n_q, n_k = cu_q[-1] + pad, cu_kk[-1] + pad
    g = torch.Generator().manual_seed(seed)
    hq = heads * group
    if strided:     # one projection's output: q, k and v side by side where the rows agree, else k and v
        both = (torch.randn(n_k, 2 * heads, dim, generator=g)).to(dtype).cuda()
        k, v = both[:, :heads], both[:, heads:]
        wide = (torch.randn(n_q, hq + 1, dim, generator=g) * q_by).to(dtype).cuda()
        q = wide[:, :hq]
        out = torch.full((n_q, hq + 2, dim), 7.0, dtype=dtype, device="cuda")[:, 1:hq + 1]
    else:
        k, v = (torch.randn(n_k, heads, dim, generator=g).to(dtype).cuda() for _ in range(2))
        q = (torch.randn(n_q, hq, dim, generator=g) * q_by).to(dtype).cuda()
        out = torch.full_like(q, 7.0)
    if pad:         # rows of no sequence may hold anything
        for x in (q, k, v):
            x[:pad] = math.nan
            x[-pad:] = math.inf
    l_out = torch.full((n_q, hq), 7.0, device="cuda") if lse else None
    dev = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    scale = 1 / math.sqrt(dim)
    H.hsa_prompt_attn(q, k, v, dev(cu_q), scale, out, cu_k=dev(cu_kk) if cu_k else None, window=window, lse=l_out)
    clean(H)
    for b, n in enumerate(lens):
        if not n:
            continue
        q0, k0, lk = cu_q[b], cu_kk[b], cu_kk[b + 1] - cu_kk[b]
        pos = torch.arange(n, device="cuda") + lk - n
        hi = (pos + 1).clamp(min=0).repeat_interleave(group)
        lo = (hi - window).clamp(min=0) if window else torch.zeros_like(hi)
        for h in range(heads):
            mine = slice(h * group, (h + 1) * group)
            rows = q[q0:q0 + n, mine].reshape(-1, dim).double()
            o, l, A, mag = D.attention(rows, k[k0:k0 + lk, h].double(), v[k0:k0 + lk, h].double(), lo, hi, scale)
            D.check(out[q0:q0 + n, mine].reshape(-1, dim), l_out[q0:q0 + n, mine].reshape(-1) if lse else None, o, l, A, mag,
                    lk, dim, dtype, f"sequence {b} head {h}")
    if pad:
        assert (out[:pad] == 7).all() and (out[-pad:] == 7).all(), "rows of no sequence were written"
        assert not lse or ((l_out[:pad] == 7).all() and (l_out[-pad:] == 7).all())
    return out


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 700])
def test_prompt_lengths(H, dim, dtype, n):
    prompt(H, [n], 2, 4, dim, dtype, seed=n, cu_k=False)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim,heads,group", [(128, 1, 1), (128, 2, 3), (64, 3, 5), (128, 1, 7), (64, 1, 16), (128, 2, 128),
                                             (64, 1, 100), (128, 4, 2), (64, 8, 1)])
def test_prompt_heads(H, dtype, dim, heads, group):
    prompt(H, [200, 3, 130], heads, group, dim, dtype, seed=group, pad=2)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("strided", [False, True])
def test_prompt_packed(H, dim, strided):
    """Many sequences, empty ones among them, padding rows that hold anything at both ends."""
    prompt(H, [5, 0, 129, 64, 1, 0, 0, 300, 17, 2, 1, 1] + [3] * 40, 2, 4, dim, BF, pad=5, strided=strided)


def test_prompt_neighbours_do_not_leak(H):
    """Infinities and NaN in one sequence stay there (they share 128-row tiles with the next one)."""
    dim, lens = 128, [70, 90, 40]
    q = torch.randn(200, 4, dim).to(BF).cuda()
    k, v = torch.randn(200, 2, dim).to(BF).cuda(), torch.randn(200, 2, dim).to(BF).cuda()
    cu = torch.tensor([0, 70, 160, 200], dtype=torch.int32).cuda()
    clean_out, out = torch.empty_like(q), torch.empty_like(q)
    H.hsa_prompt_attn(q, k, v, cu, 0.1, clean_out)
    k[70:160], v[70:160], q[70:160] = math.inf, math.nan, math.nan
    H.hsa_prompt_attn(q, k, v, cu, 0.1, out)
    clean(H)
    assert torch.equal(out[:70], clean_out[:70]) and torch.equal(out[160:], clean_out[160:])
    assert out[70:160].isnan().all() and len(lens) == 3


@pytest.mark.parametrize("past", [[100, 0, 1000], [1, 127, 128], [129, 64, 3], [0, -20, -100]])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_chunks(H, past, dim):
    """Chunks behind earlier keys, and sequences with fewer keys than queries (their first rows see nothing)."""
    prompt(H, [130, 37, 64], 2, 3, dim, HF, past=past)


@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 500, 100000])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_window(H, window, dim):
    prompt(H, [600, 1, 90], 2, 4, dim, BF, window=window)
    prompt(H, [100, 20], 1, 8, dim, BF, window=window, past=[700, 5])


def test_prompt_large_logits(H):
    """One key takes all the weight; and logits that rise along the keys, so that the maximum is raised again and again."""
    prompt(H, [300], 2, 4, 128, BF, q_by=200.0)
    n, dim = 900, 64
    k = torch.zeros(n, 1, dim)
    k[:, 0, 0] = torch.linspace(4, 0, n)           # seen from the diagonal downwards the logits grow
    k, v = k.to(HF).cuda(), torch.randn(n, 1, dim).to(HF).cuda()
    q = torch.zeros(n, 2, dim).to(HF).cuda()
    q[..., 0] = 300.0
    out, lse = torch.empty_like(q), torch.empty(n, 2, device="cuda")
    H.hsa_prompt_attn(q, k, v, torch.tensor([0, n], dtype=torch.int32).cuda(), 0.125, out, lse=lse)
    clean(H)
    hi = torch.arange(1, n + 1, device="cuda").repeat_interleave(2)
    o, l, A, mag = D.attention(q.reshape(-1, dim).double(), k[:, 0].double(), v[:, 0].double(), hi * 0, hi, 0.125)
    D.check(out.reshape(-1, dim), lse.reshape(-1), o, l, A, mag, n, dim, HF)


def test_prompt_bad_bounds_are_flagged(H):
    """Sequences whose bounds leave the tensors or descend are skipped and flagged; the others are computed."""
    q = torch.randn(100, 2, 64).to(BF).cuda()
    k, v = torch.randn(100, 2, 64).to(BF).cuda(), torch.randn(100, 2, 64).to(BF).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    want = torch.empty_like(q)
    H.hsa_prompt_attn(q, k, v, i32([0, 40, 60, 100]), 0.1, want)
    clean(H)
    for cu in ([0, 40, 60, 101], [0, 40, 30, 30], [-1, 40, 60, 100]):
        out = torch.full_like(q, 7.0)
        H.hsa_prompt_attn(q, k, v, i32(cu), 0.1, out)
        clean(H, H.HSA_FLAG_INDEX_RANGE)
        for a, b in zip(cu[:-1], cu[1:]):
            if [a, b] in ([0, 40], [40, 60], [60, 100]):
                assert torch.equal(out[a:b], want[a:b])
        if cu[-1] == 101:
            assert (out[60:] == 7).all()


@pytest.mark.parametrize("batch", [100, 129, 300, 513, 700])
def test_prompt_many_sequences(H, batch):
    """Batches past what the search for work holds in registers, and in shared memory; lengths of all sizes."""
    lens = [(7 * b * b) % 23 for b in range(batch)]
    lens[batch // 2], lens[-1] = 400, 130
    past = [(5 * b) % 40 for b in range(batch)]
    heads, group, dim = 1, 4, 64
    cu_q, cu_k = [0], [0]
    for n, o in zip(lens, past):
        cu_q.append(cu_q[-1] + n)
        cu_k.append(cu_k[-1] + n + o)
    g = torch.Generator().manual_seed(batch)
    q = torch.randn(cu_q[-1], group, dim, generator=g).to(BF).cuda()
    k, v = (torch.randn(cu_k[-1], heads, dim, generator=g).to(BF).cuda() for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    out, lse = torch.full_like(q, 7.0), torch.full((cu_q[-1], group), 7.0, device="cuda")
    H.hsa_prompt_attn(q, k, v, i32(cu_q), 0.125, out, cu_k=i32(cu_k), lse=lse)
    clean(H)
    # all sequences at once: query rows of sequence b see the keys of its own only
    seq = torch.repeat_interleave(torch.arange(batch), torch.tensor(lens)).cuda()
    pos = torch.arange(cu_q[-1], device="cuda") - i32(cu_q)[seq] + torch.tensor(past).cuda()[seq]
    lo = i32(cu_k)[seq].long()
    hi = (lo + pos + 1).repeat_interleave(group)
    lo = lo.repeat_interleave(group)
    o, l, A, mag = D.attention(q.reshape(-1, dim).double(), k[:, 0].double(), v[:, 0].double(), lo, hi, 0.125)
    D.check(out.reshape(-1, dim), lse.reshape(-1), o, l, A, mag, 500, dim, BF)
    bad = list(cu_q)
    bad[-1] = cu_q[-1] + 1                          # the last sequence leaves the tensor: skipped, the others computed
    again = torch.full_like(q, 7.0)
    H.hsa_prompt_attn(q, k, v, i32(bad), 0.125, again, cu_k=i32(cu_k))
    clean(H, H.HSA_FLAG_INDEX_RANGE)
    assert torch.equal(again[:cu_q[-2]], out[:cu_q[-2]]) and (again[cu_q[-2]:] == 7).all()


def test_prompt_without_keys_and_odd_strides(H):
    """No key rows at all; and output rows that start on 16-byte, not 32-byte, boundaries."""
    q = torch.randn(40, 4, 64).to(BF).cuda()
    none = torch.empty(0, 2, 64, dtype=BF, device="cuda")
    cu, zero = torch.tensor([0, 40], dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    out, lse = torch.full_like(q, 7.0), torch.zeros(40, 4, device="cuda")
    H.hsa_prompt_attn(q, none, none, cu, 0.1, out, cu_k=zero, lse=lse)
    clean(H)
    assert (out == 0).all() and (lse == -math.inf).all()
    k, v = torch.randn(40, 2, 64).to(BF).cuda(), torch.randn(40, 2, 64).to(BF).cuda()
    want = torch.empty_like(q)
    H.hsa_prompt_attn(q, k, v, cu, 0.1, want)
    for stride, first in ((4 * 64 + 8, 0), (4 * 64 + 8, 8), (4 * 64 + 16, 8)):
        room = torch.full((40 * stride + first,), 7.0, dtype=BF, device="cuda")
        odd = room[first:].as_strided((40, 4, 64), (stride, 64, 1))
        H.hsa_prompt_attn(q, k, v, cu, 0.1, odd)
        clean(H)
        assert torch.equal(odd, want)
        odd.fill_(7.0)
        assert (room == 7).all()                    # nothing between the rows was written


def test_waits_that_run_out(H):
    """With a wait limit of 1 ns, work whose roles wait for each other for longer than two suspensions of a wait
    (20 us each) gives up: both kernels end by themselves, the flag is set, the next calls are not affected."""
    g = torch.Generator().manual_seed(9)
    q = torch.randn(16384, 8, 128, generator=g).to(BF).cuda()
    k, v = (torch.randn(16384, 1, 128, generator=g).to(BF).cuda() for _ in range(2))
    cu = torch.tensor([0, 16384], dtype=torch.int32).cuda()
    # 200 requests that share one table row's pages: one split each, 65,536 keys for a CTA
    pk, pv, table = D.paged(1, [65536], 1, 128, 64, BF, 3)
    cache = H.PagedCache(pk.cuda(), pv.cuda(), table.expand(200, -1).contiguous().cuda())
    q_d = torch.randn(200, 5, 8, 128, generator=g).to(BF).cuda()    # 40 rows per key head
    vis = torch.full((200, 5), 65536, dtype=torch.int32).cuda()
    ws = H.new_paged_workspace(cache, 8, 5, 65536)

    def calls():
        out, out_d = torch.zeros_like(q), torch.zeros_like(q_d)
        H.hsa_prompt_attn(q, k, v, cu, 0.1, out)
        status_p = H.hsa_get_device_status()
        H.hsa_paged_attn_decode(cache, q_d, vis, 65536, 0.1, out_d, ws)
        return out, out_d, status_p, H.hsa_get_device_status()

    want = calls()
    assert want[2:] == ((0, 0), (0, 0))
    try:
        H.hsa_set_wait_limit(1)
        short = calls()
    finally:
        H.hsa_set_wait_limit(0)
    timeout = (H.STATUS_CODES["HSA_ERR_TIMEOUT"], H.HSA_FLAG_TIMEOUT)
    assert short[2:] == (timeout, timeout)
    again = calls()
    assert again[2:] == ((0, 0), (0, 0)) and torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


# ------------------------------------------------------------------------------------- together
def layer(H, cache, x, cu, start, vis, scale, out_p, out_d, q_d, ws):
    H.hsa_prompt_attn(x[:, :8], x[:, 8:10], x[:, 10:12], cu, scale, out_p)
    H.hsa_paged_cache_write(cache, x[:, 8:10], x[:, 10:12], cu=cu, start=start)
    H.hsa_paged_attn_decode(cache, q_d, vis, 400, scale, out_d, ws)


def together(dtype=BF):
    lens = [300, 1, 77]
    cu = torch.tensor([0, 300, 301, 378], dtype=torch.int32).cuda()
    k, v, table = D.paged(3, [400] * 3, 2, 128, 32, dtype, 2)
    x = torch.randn(378, 12, 128).to(dtype).cuda()
    return lens, cu, k.cuda(), v.cuda(), table.cuda(), x


def test_prompt_write_decode_together(H):
    """A layer's prompt, its pages and the next token: the token's attention over the pages is the prompt
    call's last row when its query is that row's."""
    lens, cu, k, v, table, x = together()
    cache = H.PagedCache(k, v, table)
    start = torch.zeros(3, dtype=torch.int64).cuda()
    vis = torch.tensor([[n] for n in lens], dtype=torch.int32).cuda()
    last = (cu[1:] - 1).long()
    q_d = x[last, :8][:, None].contiguous()
    out_p, out_d = torch.empty(378, 8, 128, dtype=BF, device="cuda"), torch.empty_like(q_d)
    ws = H.new_paged_workspace(cache, 8, 1, 400)
    layer(H, cache, x, cu, start, vis, 0.1, out_p, out_d, q_d, ws)
    clean(H)
    u = torch.finfo(BF).eps / 2
    a, b = out_p[last].double(), out_d[:, 0].double()
    big = x[:, 10:12].abs().max().double()
    assert ((a - b).abs() <= 4 * u * big).all()
    # the pages hold the rows
    for r, n in enumerate(lens):
        kk, _ = D.unpage(cache.k, cache.table, r, n)
        assert torch.equal(kk, x[int(cu[r]):int(cu[r]) + n, 8:10].double())


def test_captured_and_on_other_streams(H):
    """The three calls captured into a graph and replayed on new inputs, and run on a side stream, give the eager results."""
    lens, cu, k, v, table, x = together()
    start = torch.zeros(3, dtype=torch.int64).cuda()
    vis = torch.tensor([[n] for n in lens], dtype=torch.int32).cuda()
    last = (cu[1:] - 1).long()

    def eager(x, stream=None):
        cache = H.PagedCache(k.clone(), v.clone(), table)
        q_d = x[last, :8][:, None].contiguous()
        out_p, out_d = torch.zeros(378, 8, 128, dtype=BF, device="cuda"), torch.zeros_like(q_d)
        ws = H.new_paged_workspace(cache, 8, 1, 400)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            layer(H, cache, x, cu, start, vis, 0.1, out_p, out_d, q_d, ws)
        torch.cuda.synchronize()
        return out_p, out_d, cache.k

    x2 = torch.randn_like(x.float()).to(BF)
    want = [eager(x), eager(x2)]
    for a, b in zip(want[1], eager(x2, torch.cuda.Stream())):
        assert torch.equal(a, b)
    cache = H.PagedCache(k.clone(), v.clone(), table)
    xs = x.clone()
    q_d = torch.empty(3, 1, 8, 128, dtype=BF, device="cuda")
    out_p, out_d = torch.zeros(378, 8, 128, dtype=BF, device="cuda"), torch.zeros_like(q_d)
    ws = H.new_paged_workspace(cache, 8, 1, 400)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q_d.copy_(xs[last, :8][:, None])
        layer(H, cache, xs, cu, start, vis, 0.1, out_p, out_d, q_d, ws)
    for inp, ref in ((x, want[0]), (x2, want[1]), (x, want[0])):
        xs.copy_(inp)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out_p, ref[0]) and torch.equal(out_d, ref[1]) and torch.equal(cache.k, ref[2])
    clean(H)


def test_calls_at_the_same_time(H):
    """Prompts and decodes on three streams at once, each decode with its own workspace, give the bits of calls one by one."""
    g = torch.Generator().manual_seed(4)
    cu = torch.tensor([0, 900, 1500, 4000], dtype=torch.int32).cuda()
    q = torch.randn(4000, 8, 128, generator=g).to(BF).cuda()
    k, v = (torch.randn(4000, 2, 128, generator=g).to(BF).cuda() for _ in range(2))
    pk, pv, table = D.paged(30, [50 * b + 1 for b in range(30)], 2, 128, 32, BF, 3)
    cache = H.PagedCache(pk.cuda(), pv.cuda(), table.cuda())
    vis = {nq: torch.tensor([[50 * b + 1] * nq for b in range(30)], dtype=torch.int32).cuda() for nq in (1, 5)}
    q_d = {nq: torch.randn(30, nq, 14, 128, generator=g).to(BF).cuda() for nq in (1, 5)}
    ws = {nq: H.new_paged_workspace(cache, 14, nq, 1451) for nq in (1, 5)}
    work = [lambda out: H.hsa_prompt_attn(q, k, v, cu, 0.1, out)]
    work += [lambda out, nq=nq: H.hsa_paged_attn_decode(cache, q_d[nq], vis[nq], 1451, 0.1, out, ws[nq]) for nq in (1, 5)]
    like = [q, q_d[1], q_d[5]]
    want = [torch.empty_like(x) for x in like]
    for w, x in zip(work, want):
        w(x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(5):
        got = [torch.zeros_like(x) for x in like]
        torch.cuda.synchronize()
        for _ in range(4):
            for w, x, s in zip(work, got, streams):
                with torch.cuda.stream(s):
                    w(x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    clean(H)


def test_same_inputs_same_bits(H):
    """Splits are joined in their order: the same call gives the same bits."""
    first = decode(H, 2, 1, 2, 8, 128, 64, BF, BF, [[3000], [1234]])
    for _ in range(3):
        assert torch.equal(first, decode(H, 2, 1, 2, 8, 128, 64, BF, BF, [[3000], [1234]]))
