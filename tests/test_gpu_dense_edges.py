"""Dense attention calls on the GPU where positions, weights and bounds leave the ordinary: queries
further apart than their window, weights that reach over many orders, sequences that overlap, pools
past 2^31 bytes. Bounds: tests/dense.py, with what is added here derived where it is used."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


# ------------------------------------------------------------------------------------- far queries
@pytest.mark.parametrize("kv,qt", [(BF, BF), (HF, HF), (F8, BF)])
@pytest.mark.parametrize("dim,heads,group,page", [(128, 2, 4, 16), (64, 1, 16, 48), (128, 1, 9, 64), (64, 2, 12, 32), (128, 1, 42, 128)])
@pytest.mark.parametrize("window", [1, 15, 64, 130, 700])
def test_decode_queries_further_apart_than_the_window(H, kv, qt, dim, heads, group, page, window):
    """Positions between the windows of a request's queries are seen by none: whatever the pools hold there is not
    used, and table entries that only they need are not pages."""
    vis = [[40, 2000, 900], [300, 0, 310], [1, 1500, 1]]
    batch, nq, longest = 3, 3, [max(r) for r in vis]
    k, v, table = D.paged(batch, longest, heads, dim, page, kv, window)
    seen = torch.zeros(k.shape[0], page, dtype=torch.bool)
    for b, r in enumerate(vis):
        mine = torch.zeros(-(-longest[b] // page) * page, dtype=torch.bool)
        for x in r:
            mine[max(0, x - window):x] = True
        for i, held in enumerate(mine.view(-1, page)):
            seen[table[b, i].long()] = held
            if not held.any():
                table[b, i] = (-1, 1 << 20)[i & 1]
    raw = torch.uint8 if kv == F8 else torch.int16
    bad = torch.tensor([math.nan] * 3 if kv == F8 else [math.nan, math.inf, -math.inf]).to(kv)
    for x in (k, v):
        fill = bad.view(raw)[torch.randint(0, 3, x.shape, generator=torch.Generator().manual_seed(1))]
        x.view(raw).copy_(torch.where(seen[:, None, :, None], x.view(raw), fill))
    k, v, table = k.cuda(), v.cuda(), table.cuda()
    q = (torch.randn(batch, nq, heads * group, dim, generator=torch.Generator().manual_seed(2)) * 2).to(qt).cuda()
    scale = 1 / math.sqrt(dim)
    # the bound as it is, and one that cuts the length into many splits
    for most in (2000, 30000):
        wide = torch.cat([table, table.new_full((batch, -(-most // page)), -1)], 1)
        cache = H.PagedCache(k, v, wide)
        out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
        H.hsa_paged_attn_decode(cache, q, i32(vis), most, scale, out, H.new_paged_workspace(cache, heads * group, nq, most),
                                window=window, lse=lse)
        clean(H)
        for b in range(batch):
            kk, vv = (D.unpage(x, table, b, longest[b])[0] for x in (k, v))
            hi = i32(vis[b]).repeat_interleave(group)
            lo = (hi - window).clamp(min=0)
            for h in range(heads):
                mine = slice(h * group, (h + 1) * group)
                o, l, A, mag = D.attention(q[b, :, mine].reshape(-1, dim).double(), kk[:, h], vv[:, h], lo, hi, scale)
                D.check(out[b, :, mine].reshape(-1, dim), lse[b, :, mine].reshape(-1), o, l, A, mag, longest[b], dim,
                        BF if kv == BF else HF, f"window {window} bound {most} request {b} head {h}")


# ------------------------------------------------------------------------------------- a long tail of weights
def tail(n, heads, dim, kv, at, gap):
    """Keys whose logits are alike (within about 0.5) but for those at `at`, `gap` higher and with v = 0, and a query row."""
    g = torch.Generator().manual_seed(n)
    k, v = torch.randn(n, heads, dim, generator=g), 1 + 0.25 * torch.randn(n, heads, dim, generator=g)
    k[..., 0] = 0
    k[at] = 0
    k[at, :, 0] = 4.0
    v[at] = 0
    q = torch.full((dim,), 0.5)
    q[0] = gap * math.sqrt(dim) / 4
    return q, k.to(kv), v.to(kv)


def with_floor(A, n, v, p_type, o_type, lse, top):
    """A, raised so that the bound of tests/dense.py gains the absolute part of the weights' rounding: an f16 weight below
    2^-14 is off by up to 2^-25, in units where the row's largest weight is 2^7 at least and their sum 2^7 exp(lse - top)
    with it, for each of n keys. The bound multiplies A by u_p + u_o + 2 n 2^-23 and more."""
    if p_type != HF:
        return A
    rel = 2.0 ** -11 + torch.finfo(o_type).eps / 2 + 2 * n * 2.0 ** -23
    return A + n * 2.0 ** -32 * torch.exp(top - lse)[:, None] * v.abs().max() / rel


@pytest.mark.parametrize("gap", [14.0, 16.0, 17.0, 17.4])
@pytest.mark.parametrize("kv,qt", [(HF, HF), (F8, HF), (F8, BF), (BF, BF)])
@pytest.mark.parametrize("dim,group", [(128, 8), (64, 16), (128, 28), (64, 64)])
def test_decode_long_tail(H, kv, qt, dim, group, gap):
    """A few keys far above 65,529 alike: the tail's weights are 2^-20 and less, and what they bring together is kept. The
    high keys stand where each warp and each stream of a CTA meets them first."""
    n, heads, page, batch = 65536, 4, 64, 128
    at = [0, 16, 32, 48, n // 4, n // 2, 3 * n // 4]
    q, k, v = tail(n, heads, dim, kv, at, gap)
    pages = n // page
    k, v = (x.view(torch.uint8 if kv == F8 else kv).view(pages, page, heads, -1).transpose(1, 2).contiguous().view(kv).cuda() for x in (k, v))
    table = torch.arange(pages, dtype=torch.int32).cuda().repeat(batch, 1)
    q = q.to(qt).cuda().expand(batch, 1, heads * group, dim).contiguous()
    cache = H.PagedCache(k, v, table)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    vis = torch.full((batch, 1), n, dtype=torch.int32, device="cuda")
    scale = 1 / math.sqrt(dim)
    H.hsa_paged_attn_decode(cache, q, vis, n, scale, out, H.new_paged_workspace(cache, heads * group, 1, n), lse=lse)
    clean(H)
    kk, vv = (D.unpage(x, table, 0, n)[0] for x in (k, v))
    hi = torch.full((1,), n, device="cuda")
    p_type = BF if kv == BF else HF
    for h in range(heads):
        row = q[0, 0, h * group][None].double()
        o, l, A, mag = D.attention(row, kk[:, h], vv[:, h], hi * 0, hi, scale)
        A = with_floor(A, n, vv, p_type, qt, l, (row @ kk[:, h].T).max() * scale)
        for r in (h * group, (h + 1) * group - 1):
            D.check(out[0, :1, r], lse[0, :1, r], o, l, A, mag, n, dim, p_type, f"head {h}")
    assert torch.equal(out[0], out[-1]) and torch.equal(lse[0], lse[-1])


@pytest.mark.parametrize("gap", [14.0, 16.0, 17.0, 17.4])
@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_long_tail(H, dim, dtype, gap):
    """The same for the last rows of a prompt, whose key tiles are met from the diagonal downwards."""
    n, group, last = 16384, 4, 256
    q, k, v = tail(n, 1, dim, dtype, [n - last], gap)
    q = q.to(dtype).cuda().expand(last, group, dim).contiguous()
    k, v = k.cuda(), v.cuda()
    out, lse = torch.empty_like(q), torch.empty(last, group, device="cuda")
    scale = 1 / math.sqrt(dim)
    H.hsa_prompt_attn(q, k, v, i32([0, last]), scale, out, cu_k=i32([0, n]), lse=lse)
    clean(H)
    hi = torch.arange(n - last + 1, n + 1, device="cuda").repeat_interleave(group)
    o, l, A, mag = D.attention(q.reshape(-1, dim).double(), k[:, 0].double(), v[:, 0].double(), hi * 0, hi, scale)
    top = (q[0, 0].double() @ k[:, 0].double().T).max() * scale        # every row sees it
    D.check(out.reshape(-1, dim), lse.reshape(-1), o, l, with_floor(A, n, v.double(), dtype, dtype, l, top), mag, n, dim, dtype)


# ------------------------------------------------------------------------------------- sequences that overlap
@pytest.mark.parametrize("batch", [5, 40, 600])
@pytest.mark.parametrize("group", [1, 4])
def test_prompt_sequences_that_overlap(H, batch, group):
    """Bounds that go back and start again: what an earlier sequence has is not given out twice, every other sequence is
    computed, and the flag is set."""
    n, dim = 1500, 64
    g = torch.Generator().manual_seed(batch)
    q = torch.randn(n, group, dim, generator=g).to(BF).cuda()
    k, v = (torch.randn(2 * n, 1, dim, generator=g).to(BF).cuda() for _ in range(2))
    # [0, 1000) over and over, each time with other keys, then [1000, 1500)
    cu_q = [0, 1000] * (batch // 2) + [1000] * (batch % 2) + [n]
    assert len(cu_q) == batch + 1
    cu_k = [0, 1000] + [1200 + b for b in range(batch - 2)] + [2 * n]
    out, lse = torch.full_like(q, 7.0), torch.full((n, group), 7.0, device="cuda")
    H.hsa_prompt_attn(q, k, v, i32(cu_q), 0.125, out, cu_k=i32(cu_k), lse=lse)
    clean(H, H.HSA_FLAG_INDEX_RANGE)
    first = cu_k[batch - 1]
    for q0, q1, k0, k1 in ((0, 1000, 0, 1000), (1000, n, first, 2 * n)):
        hi = (torch.arange(q1 - q0, device="cuda") + (k1 - k0) - (q1 - q0) + 1).repeat_interleave(group)
        o, l, A, mag = D.attention(q[q0:q1].reshape(-1, dim).double(), k[k0:k1, 0].double(), v[k0:k1, 0].double(), hi * 0, hi, 0.125)
        D.check(out[q0:q1].reshape(-1, dim), lse[q0:q1].reshape(-1), o, l, A, mag, k1 - k0, dim, BF, f"rows from {q0}")


def test_prompt_sequences_that_share_keys(H):
    """Bounds of the keys that go back: the sequence whose own keys descend is skipped, those around it are computed
    from the same keys."""
    n, dim = 64, 64
    g = torch.Generator().manual_seed(3)
    q = torch.randn(3 * n, 2, dim, generator=g).to(HF).cuda()
    k, v = (torch.randn(2 * n, 1, dim, generator=g).to(HF).cuda() for _ in range(2))
    out = torch.full_like(q, 7.0)
    H.hsa_prompt_attn(q, k, v, i32([0, n, 2 * n, 3 * n]), 0.125, out, cu_k=i32([0, 2 * n, 0, 2 * n]))
    clean(H, H.HSA_FLAG_INDEX_RANGE)
    for q0 in (0, 2 * n):
        hi = (torch.arange(n, device="cuda") + n + 1).repeat_interleave(2)
        o, l, A, mag = D.attention(q[q0:q0 + n].reshape(-1, dim).double(), k[:, 0].double(), v[:, 0].double(), hi * 0, hi, 0.125)
        D.check(out[q0:q0 + n].reshape(-1, dim), None, o, l, A, mag, 2 * n, dim, HF, f"rows from {q0}")
    assert (out[n:2 * n] == 7).all()


# ------------------------------------------------------------------------------------- tiles of query rows
@pytest.mark.parametrize("kv", [BF, HF])
@pytest.mark.parametrize("dim,group,nq", [(128, 7, 5), (64, 13, 2), (128, 42, 8), (64, 33, 1), (128, 65, 3), (64, 5, 8)])
def test_decode_tiles_of_queries(H, kv, dim, group, nq):
    """Requests of 26 to 336 rows per key head, one of them with queries that are NaN: it is the only one that notices."""
    vis = [[500 - i for i in range(nq)], [64] * nq, [1000] * nq]
    k, v, table = D.paged(3, [500, 64, 1000], 2, dim, 32, kv, group)
    cache = H.PagedCache(k.cuda(), v.cuda(), table.cuda())
    q = torch.randn(3, nq, 2 * group, dim, generator=torch.Generator().manual_seed(nq)).to(kv).cuda()
    q[1] = math.nan
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
    H.hsa_paged_attn_decode(cache, q, i32(vis), 1000, 0.1, out, H.new_paged_workspace(cache, 2 * group, nq, 1000), lse=lse)
    clean(H)
    assert out[1].isnan().all()
    for b in (0, 2):
        kk, vv = (D.unpage(x, cache.table, b, max(vis[b]))[0] for x in (cache.k, cache.v))
        hi = i32(vis[b]).repeat_interleave(group)
        for h in range(2):
            mine = slice(h * group, (h + 1) * group)
            o, l, A, mag = D.attention(q[b, :, mine].reshape(-1, dim).double(), kk[:, h], vv[:, h], hi * 0, hi, 0.1)
            D.check(out[b, :, mine].reshape(-1, dim), lse[b, :, mine].reshape(-1), o, l, A, mag, max(vis[b]), dim, kv, f"request {b}")


# ------------------------------------------------------------------------------------- large pools
@pytest.mark.parametrize("dtype", [BF, HF])
def test_decode_many_rows_past_2_31_bytes(H, dtype):
    """The kernel for many rows on pages that start past 2^31 bytes and 2^31 elements of their pools."""
    heads, page, dim, group, n = 2, 64, 128, 40, 311
    pages = (2 ** 31 + 2 ** 28) // (heads * page * dim)             # elements
    need = -(-n // page)
    g = torch.Generator().manual_seed(7)
    pools = []
    for _ in range(2):
        pool = torch.zeros(pages, heads, page, dim, dtype=dtype, device="cuda")
        pool[-need:] = torch.randn(need, heads, page, dim, generator=g).to(dtype).cuda()
        pools.append(pool)
    q = torch.randn(1, 1, heads * group, dim, generator=g).to(dtype).cuda()
    outs = []
    for k, v, first in ((*pools, pages - need), (*(x[-need:].clone() for x in pools), 0)):
        cache = H.PagedCache(k, v, i32([list(range(first, first + need))]))
        out = torch.empty_like(q)
        H.hsa_paged_attn_decode(cache, q, i32([[n]]), n, 0.1, out, H.new_paged_workspace(cache, heads * group, 1, n))
        outs.append(out)
    clean(H)
    assert torch.equal(*outs) and outs[0].isfinite().all()


# ------------------------------------------------------------------------------------- E4M3 codes
@pytest.mark.parametrize("src", [BF, HF])
@pytest.mark.parametrize("scale", [0.875, 7.0, 0.3, 0.0234375, 2.0 ** -100, 2.0 ** 100])
def test_write_every_value_to_e4m3(H, src, scale):
    """All 65,536 values of a 16-bit type: the code of the fp32 product with the scale's reciprocal, which is the nearest to
    x / scale but where that lies in the middle of two E4M3 values, up to the product's two roundings (2^-23)."""
    heads, dim, page = 8, 128, 16
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(src).view(64, heads, dim).cuda()
    k, v, table = D.paged(1, [64], heads, dim, page, F8, 4)
    cache = H.PagedCache(k.cuda(), v.cuda(), table.cuda(), scale, 1.0)
    H.hsa_paged_cache_write(cache, x, x)
    clean(H)
    got = D.unpage(cache.k, cache.table, 0, 64)[0]
    inv = 1 / torch.tensor(scale, dtype=torch.float32, device="cuda")
    y = x.float() * inv
    want = y.clamp(-448, 448).to(F8).double()
    nan = x.isnan()
    assert torch.equal(got.isnan(), nan) and torch.equal(got[~nan], want[~nan])
    true = (x.double() / torch.tensor(scale, dtype=torch.float32).double().item())[~nan].clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(true.abs().clamp(min=2.0 ** -6))) - 3)
    off = (got[~nan] - true).abs()
    assert (off <= step / 2 + true.abs() * 2.0 ** -23).all()


def test_write_beside_a_tie(H):
    """The example of the declaration: 203 / 0.875 is 232, in the middle of 224 and 240; the product lies above it."""
    k, v, table = D.paged(1, [16], 1, 64, 16, F8, 4)
    cache = H.PagedCache(k.cuda(), v.cuda(), table.cuda(), 0.875, 1.0)
    x = torch.full((1, 1, 64), 203.0, dtype=BF, device="cuda")
    H.hsa_paged_cache_write(cache, x, x)
    clean(H)
    kk, vv = (D.unpage(p, cache.table, 0, 1)[0] for p in (cache.k, cache.v))
    assert (kk == 240).all() and (vv == 208).all()      # 203 alone goes to 208: steps of 16
