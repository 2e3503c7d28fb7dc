"""The calls of a speculative step over a paged cache on the GPU against plain 64-bit forms: rotated append, read, attention over
4-bit pages, verification of drafts, and all of them together.

Bounds (u = torch.finfo(t).eps / 2 of the 16-bit type). A rotated value x cos - y sin is a sum of two products in fp32: the sines are
off by at most 2^-23 (an ulp of sincospif, and the angle's own rounding: an eighth of a turn at most to 2^-24 of it), each
product and the sum by 2^-24 of theirs, and the angle by 2^-52 of its turns: together at most
  off = (2^-21 + 2^-49 |pos inv_freq|) (|x| + |y|), and u of the result when it is rounded to 16 bits.
A value that goes to 8 or 4 bits is multiplied by the fp32 reciprocal of its scale (2^-24 twice): 2^-22 of it more; E2M1
divides by the group's scale in fp32 (within the same). Codes are monotone in their value, so they must lie between
those of value - off and value + off."""
import math

import pytest
import torch

from tests import dense as D
from tests import four

pytestmark = pytest.mark.gpu

BF, HF, F32, F8, F4 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, "e2m1"


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


def starts(counts):
    return i32([0] + torch.tensor(counts).cumsum(0).tolist())


def cache_of(H, longest, heads, dim, page, kv, seed, scales=(1.0, 1.0), spare=2):
    """A cache with values everywhere; a request's pages are in any order."""
    k, v, table = D.paged(len(longest), longest, heads, dim, page, F32 if kv == F4 else kv, seed, spare)
    if kv != F4:
        return H.PagedCache(k.cuda(), v.cuda(), table.cuda(), *scales)
    (k, ks), (v, vs) = four.pack(k.cuda(), True), four.pack(v.cuda(), False)
    return H.PagedCache(k, v, table.cuda(), *scales, ks, vs)


def copies(c):
    return [None if t is None else t.clone() for t in (c.k, c.v, c.k_s, c.v_s)]


def rows_at(c, b, pos):
    """(where, row) of positions of request b."""
    return c.table[b].long()[pos // c.page_size], pos % c.page_size


# --------------------------------------------------------------------------------------- append
def append(H, counts, past, heads, group, dim, page, src, kv, rotary, at, halves, scales=(1.0, 1.0), in_place=False, pad=0, seed=0, cu=True,
           inv_freq=None):
    """Append and compare every written place; everything else stays as it was."""
    g = torch.Generator().manual_seed(seed)
    n = sum(counts) + pad
    cache = cache_of(H, [a + b for a, b in zip(counts, past)], heads, dim, page, kv, seed, scales)
    rows = torch.randn(n, heads * (group + 2) + 1, dim, generator=g).to(src).cuda()
    q, k, v = rows[:, :heads * group], rows[:, heads * group:heads * (group + 1)], rows[:, heads * (group + 1):heads * (group + 2)]
    keep = rows.clone()
    q_in = keep[:, :heads * group]
    out = q if in_place else torch.full((n, heads * group + 2, dim), 7.0, dtype=src, device="cuda")[:, :heads * group]
    if inv_freq is None:
        inv_freq = (160000.0 ** (-torch.arange(rotary // 2) / max(1, rotary // 2))).float()
    inv_freq = inv_freq.cuda()
    before = copies(cache)
    start = torch.tensor(past, dtype=torch.int64).cuda()
    H.hsa_paged_cache_append(cache, k, v, inv_freq if rotary else None, q=q if group else None, q_out=out if group else None,
                             cu=starts(counts) if cu else None, start=start, rotary_at=at,
                             pairs=H.HSA_ROPE_HALVES if halves else H.HSA_ROPE_NEIGHBOURS)
    clean(H)
    u = torch.finfo(src).eps / 2
    touched = [None if t is None else torch.zeros(t.shape[:3], dtype=torch.bool, device="cuda") for t in before]
    t0 = 0
    for b, count in enumerate(counts):
        pos = torch.arange(past[b], past[b] + count, device="cuda")
        mine = slice(t0, t0 + count)
        t0 += count
        if not count:
            continue
        turns = 2.0 ** -21 + 2.0 ** -49 * pos.double()[:, None, None] * float(inv_freq.max() if rotary else 0)
        if group:
            want, size = four.rotate(q_in[mine], pos, inv_freq, at, halves)
            off = (out[mine].double() - want).abs()
            bound = u * want.abs() + turns * size * (1 + u) + torch.finfo(src).smallest_normal * u * 2
            assert (off <= bound).all(), f"q of request {b}: {(off / bound).max()} times its bound"
            assert torch.equal(out[mine].double()[size == 0], want[size == 0])
        where, row = rows_at(cache, b, pos)
        for pool, scale_pool, x, scale, keys in ((cache.k, cache.k_s, k, scales[0], True), (cache.v, cache.v_s, v, scales[1], False)):
            want, size = four.rotate(x[mine], pos, inv_freq, at, halves) if keys else (x[mine].double(), torch.zeros_like(x[mine], dtype=torch.float64))
            got = pool.view(torch.uint8 if pool.element_size() == 1 else pool.dtype)[where, :, row]
            off = turns * size
            if kv in (F8, F4):
                off = (off + (2.0 ** -22 * want.abs() if scale != 1 or keys else 0)) / scale
                want = want / scale
            if kv == F4:
                four.check_group(got, scale_pool[where, :, row], want, off, keys)
            elif kv == F8:
                lo, hi = ((want + s * off).clamp(-448, 448).float().to(F8).double() for s in (-1, 1))
                got = got.view(F8).double()
                slack = 2.0 ** -24 * want.abs()          # the bounds' own rounding to fp32
                assert ((got >= lo - slack) & (got <= hi + slack)).all()
            else:
                bound = u * want.abs() + off * (1 + u) + torch.finfo(src).smallest_normal * u * 2
                assert ((got.double() - want).abs() <= bound).all()
                assert torch.equal(got.double()[size == 0], want[size == 0])
        for t in touched:
            if t is not None:
                t[where, :, row] = True
    for new, old, t in zip(copies(cache), before, touched):
        if new is not None:
            raw = torch.uint8 if new.element_size() == 1 else torch.int16
            assert torch.equal(new.view(raw)[~t], old.view(raw)[~t]), "a place that no row belongs to changed"
    if in_place:
        assert torch.equal(rows[:, heads * group:], keep[:, heads * group:]) and torch.equal(rows[t0:], keep[t0:])
    else:
        assert torch.equal(rows, keep)
        if group:
            whole = out._base if out._base is not None else out
            assert (whole[t0:] == 7).all() and (whole[:, heads * group:] == 7).all()
    return cache, out


@pytest.mark.parametrize("src,kv", [(BF, BF), (HF, HF), (BF, F8), (HF, F8), (BF, F4), (HF, F4)])
@pytest.mark.parametrize("heads,group,dim,page,rotary,at,halves,counts,past", [
    (1, 1, 64, 16, 64, 0, True, [1], [0]), (2, 4, 128, 32, 128, 0, True, [1, 1, 1], [0, 31, 700]),
    (3, 7, 128, 48, 64, 0, False, [33, 0, 5], [15, 4, 0]), (8, 4, 128, 64, 64, 64, True, [77], [100]),
    (5, 3, 64, 80, 32, 16, False, [40, 1], [3, 79]), (16, 1, 64, 16, 32, 32, True, [9, 9], [0, 16]),
    (2, 2, 128, 256, 96, 16, False, [300], [1]), (1, 33, 128, 16, 0, 0, True, [3, 4], [9, 9]), (4, 0, 64, 16, 64, 0, False, [70], [2])])
def test_append(H, src, kv, heads, group, dim, page, rotary, at, halves, counts, past):
    append(H, counts, past, heads, group, dim, page, src, kv, rotary, at, halves, scales=(0.5, 0.375) if kv in (F8, F4) else (1.0, 1.0),
           pad=3, seed=heads + dim)


@pytest.mark.parametrize("kv", [BF, F4])
@pytest.mark.parametrize("halves", [True, False])
def test_append_in_place_and_equal_shares(H, kv, halves):
    append(H, [20, 20], [5, 50], 2, 3, 128, 16, BF, kv, 64, 32, halves, in_place=True, cu=False)
    append(H, [2], [7], 2, 40, 64, 16, BF, kv, 64, 0, halves, in_place=True)


@pytest.mark.parametrize("kv", [HF, F4])
def test_append_far_positions(H, kv):
    """Angles of positions up to 2^31 and frequencies up to several turns per position."""
    src, page, heads, dim = HF, 4096, 1, 64
    inv = torch.tensor([1.0, 0.7, 6.5, 100.0, 0.01, 2.0 ** -20, 3.14159274, 0.0] * 4).float().cuda()
    k = torch.randn(8, heads, dim).to(src).cuda()
    pools = [torch.zeros(2, heads, page, dim if kv == HF else dim // 2, dtype=HF if kv == HF else torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(2, heads, page, dim // 16, dtype=torch.uint8, device="cuda") for _ in range(2)] if kv == F4 else (None, None)
    table = torch.full((1, (1 << 31) // page - 1), -1, dtype=torch.int32, device="cuda")
    for first in (0, 123456789, (1 << 31) - 3 * page):
        table[:, first // page:first // page + 2] = i32([1, 0])
        cache = H.PagedCache(*pools, table, 1.0, 1.0, *scales)
        q = torch.empty_like(k)
        H.hsa_paged_cache_append(cache, k, k, inv, q=k, q_out=q, start=torch.tensor([first]).cuda())
        clean(H)
        pos = torch.arange(first, first + 8, device="cuda")
        want, size = four.rotate(k, pos, inv, 0, True)
        turns = torch.cat((inv, inv)).double() * pos.double()[:, None]
        bound = 2.0 ** -11 * want.abs() + (2.0 ** -21 + 2.0 ** -49 * turns[:, None]) * size * 1.001 + 2.0 ** -25
        assert ((q.double() - want).abs() <= bound).all()
        where, row = rows_at(cache, 0, pos)
        if kv == HF:
            assert torch.equal(cache.k[where, :, row], q)
        else:
            four.check_group(cache.k[where, :, row], cache.k_s[where, :, row], want, (2.0 ** -20 + 2.0 ** -49 * turns[:, None]) * size, True)


def test_append_out_of_range_rows_are_flagged(H):
    """Positions without a place keep their pages' neighbours and still have rotated queries."""
    inv = torch.ones(32, device="cuda")
    for kv in (BF, F8, F4):
        cache = cache_of(H, [64, 64], 2, 64, 16, kv, 3)
        cache.table[1, 1] = -1
        cache.table[1, 2] = 1 << 30
        x = torch.randn(60, 2, 64).to(BF).cuda()
        q, before = torch.zeros_like(x), copies(cache)
        H.hsa_paged_cache_append(cache, x, x, inv, q=x, q_out=q, cu=i32([0, 10, 60]), start=torch.tensor([60, 14]).cuda())
        clean(H, H.HSA_FLAG_WRITE_RANGE)
        for b, first, count in ((0, 60, 10), (1, 14, 50)):
            pos = torch.arange(first, first + count, device="cuda")
            want, _ = four.rotate(x[:10] if b == 0 else x[10:], pos, inv, 0, True)
            got = q[:10] if b == 0 else q[10:]
            assert ((got.double() - want).abs() <= 2.0 ** -7 * 4).all() and (got != 0).any()
        good = torch.zeros(before[0].shape[0], 16, dtype=torch.bool, device="cuda")
        for b, pos in ((0, range(60, 64)), (1, (14, 15, *range(48, 64)))):
            for t in pos:
                good[cache.table[b, t // 16].long(), t % 16] = True
        for new, old in zip(copies(cache), before):
            if new is not None:
                raw = torch.uint8 if new.element_size() == 1 else torch.int16
                changed = (new.view(raw) != old.view(raw)).flatten(3).any(-1).any(1)
                assert not (changed & ~good).any()
        H.hsa_paged_cache_append(cache, x[:4], x[:4], inv, start=torch.tensor([-1, -9]).cuda())
        clean(H, H.HSA_FLAG_WRITE_RANGE)


@pytest.mark.parametrize("src", [BF, HF])
def test_write_to_four_bits(H, src):
    """hsa_paged_cache_write to 4-bit pages: exact codes and scales where the pool's scale is 1; zeros, ties, infinities, NaN."""
    heads, dim, page = 2, 128, 32
    cache = cache_of(H, [200], heads, dim, page, F4, 1)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(200, heads, dim, generator=g) * 2.0 ** torch.randint(-12, 12, (200, heads, dim // 16), generator=g).repeat_interleave(16, -1)
    x[0] = 0
    x[1, :, 16:32] = -0.0
    x[2] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]).repeat(16)           # every tie at scale 1
    x[3] = -x[2]
    x[4, :, :16] = torch.linspace(0, 2.0 ** -9, 16)                                          # below the smallest scale
    x[5, :, :16] = 60000.0                                                                   # above the largest
    x = x.to(src)
    y = x.clone()
    y[6, :, 3], y[6, :, 40], y[7, :, 100] = math.inf, -math.inf, math.nan
    H.hsa_paged_cache_write(cache, y.cuda(), y.cuda())
    clean(H)
    where, row = rows_at(cache, 0, torch.arange(200).cuda())
    for pool, scales, keys in ((cache.k, cache.k_s, True), (cache.v, cache.v_s, False)):
        b, s = pool[where, :, row], scales[where, :, row]
        same = torch.tensor([t for t in range(200) if t not in (6, 7)]).cuda()
        wb, ws = four.pack(x.cuda(), keys)
        assert torch.equal(s[same], ws[same]) and torch.equal(b[same], wb[same])
        c = four.codes(b, keys)
        assert (s[6, :, 0] == 0x7E).all() and (c[6, :, 3] == 7).all() and (s[6, :, 2] == 0x7E).all() and (c[6, :, 40] == -7).all()
        assert (c[6, :, 4:16] == 0).all()                                                    # beside infinity nothing is left
        assert (s[7, :, 6] == 0x7F).all() and torch.equal(s[7, :, :6], ws[7, :, :6])


# ----------------------------------------------------------------------------------------- read
@pytest.mark.parametrize("kv,dst", [(BF, BF), (HF, HF), (F8, BF), (F8, HF), (F4, BF), (F4, HF)])
@pytest.mark.parametrize("heads,dim,page,counts,start", [
    (1, 64, 16, [1], [0]), (8, 128, 64, [100, 0, 37], [0, 5, 700]), (3, 64, 48, [65], [15]), (5, 128, 16, [31, 33], [1, 16]),
    (16, 64, 256, [300], [40]), (2, 128, 32, [9, 9], [3, 0])])
def test_read(H, kv, dst, heads, dim, page, counts, start):
    scales = (0.5, 4.0) if kv in (F8, F4) else (1.0, 1.0)
    cache = cache_of(H, [a + b for a, b in zip(counts, start)], heads, dim, page, kv, dim + heads, scales)
    n = sum(counts)
    rows = torch.full((n + 4, 2 * heads + 1, dim), 7.0, dtype=dst, device="cuda")
    equal = len(set(counts)) == 1
    for cu in ([starts(counts)] + [None] * equal):
        m = n + 4 if cu is not None else n
        rows.fill_(7.0)
        H.hsa_paged_cache_read(cache, rows[:m, :heads], rows[:m, heads:2 * heads], cu=cu, start=torch.tensor(start).cuda())
        clean(H)
        t0 = 0
        for b, count in enumerate(counts):
            if count:
                where, row = rows_at(cache, b, torch.arange(start[b], start[b] + count).cuda())
                for i, (pool, s, scale, keys) in enumerate(((cache.k, cache.k_s, scales[0], True), (cache.v, cache.v_s, scales[1], False))):
                    if kv == F4:
                        want = four.unpack(pool[where, :, row], s[where, :, row], keys)
                    else:
                        want = pool.view(torch.uint8 if kv == F8 else kv)[where, :, row].view(kv).double()
                    assert torch.equal(rows[t0:t0 + count, i * heads:(i + 1) * heads], (want * scale).to(dst))
            t0 += count
        assert (rows[n:] == 7).all() and (rows[:, 2 * heads] == 7).all()


def test_read_out_of_range_rows_are_flagged(H):
    for kv in (BF, F8, F4):
        cache = cache_of(H, [64, 64], 2, 64, 16, kv, 3)
        cache.table[1, 1] = -1
        k, v = (torch.full((60, 2, 64), 7.0, dtype=BF, device="cuda") for _ in range(2))
        H.hsa_paged_cache_read(cache, k, v, cu=i32([0, 10, 50]), start=torch.tensor([60, 14]).cuda())
        clean(H, H.HSA_FLAG_INDEX_RANGE)
        left = [*range(4, 10), *range(12, 28), *range(50, 60)]           # past the table, on the bad page, padding
        for x in (k, v):
            assert (x[left] == 7).all() and not (x[[0, 3, 10, 11, 28, 49]] == 7).all(-1).any()


# --------------------------------------------------------------------------------------- decode
def decode(H, batch, nq, heads, group, dim, page, qt, vis, window=0, max_vis=None, seed=0, scales=(1., 1.), q_by=2.0, table_edit=None, flags=0,
           lse=True, spread=False):
    """Attention over 4-bit pages against the 64-bit form; what no query sees holds NaN scales."""
    longest = [max(r) for r in vis]
    k, v, table = D.paged(batch, longest, heads, dim, page, F32, seed)
    if spread:                                           # groups of very different size
        g = torch.Generator().manual_seed(seed + 7)
        k, v = (x * 2.0 ** torch.randint(-6, 4, (*x.shape[:3], dim // 16), generator=g).repeat_interleave(16, -1) for x in (k, v))
    (k, ks), (v, vs) = four.pack(k.cuda(), True), four.pack(v.cuda(), False)
    seen = torch.zeros(k.shape[0], page, dtype=torch.bool)
    for b, r in enumerate(vis):
        for x in r:
            for t in range(max(0, x - window) if window else 0, x):
                seen[table[b, t // page].long(), t % page] = True
    hidden = ~seen[:, None, :, None].cuda()
    for codes, s in ((k, ks), (v, vs)):
        s.masked_fill_(hidden, 0x7F)
        codes.copy_(torch.where(hidden, torch.randint(0, 256, codes.shape, device="cuda", dtype=torch.uint8), codes))
    if table_edit:
        table_edit(table)
    if max_vis is not None:
        table = torch.cat([table, table.new_full((batch, -(-max_vis // page)), -1)], 1)
    cache = H.PagedCache(k, v, table.cuda(), *scales, ks, vs)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn(batch, nq, heads * group, dim, generator=g) * q_by).to(qt).cuda()
    max_vis = max(longest) if max_vis is None else max_vis
    out = torch.full_like(q, 7.0)
    l_out = torch.full(q.shape[:3], 7.0, device="cuda") if lse else None
    ws = H.new_paged_workspace(cache, heads * group, nq, max_vis)
    ws.fill_(0xFF)
    scale = 1 / math.sqrt(dim)
    H.hsa_paged_attn_decode(cache, q, i32(vis), max_vis, scale, out, ws, window=window, lse=l_out)
    clean(H, flags)
    check_decode(cache, q, vis, window, scale, out, l_out, group)
    return out


def with_floor(A, rows, k, v, lo, hi, scale, ok, lse, o_type):
    """A, raised so that the bound of tests/dense.py gains the absolute part of the weights' rounding: an f16 weight below 2^-14 is
    off by up to 2^-25, in units where the row's largest is 2^7 at least, so key j by 2^-32 exp(top - lse) |v_j|. Values in 4
    bits are often exactly 0, so that keys far below the row's largest may be all that a dim has. The bound multiplies
    A by u_p + u_o and more."""
    if not k.shape[0]:
        return A
    at = torch.arange(k.shape[0], device=k.device)
    seen = (at[None] >= lo[:, None]) & (at[None] < hi[:, None]) & ok[None]
    top = ((rows @ k.T) * scale).masked_fill(~seen, -math.inf).amax(-1)
    part = torch.exp(top - lse).nan_to_num(0)[:, None] * (seen.double() @ v.abs())
    return A + 2.0 ** -32 * part / (2.0 ** -11 + torch.finfo(o_type).eps / 2)


def check_decode(cache, q, vis, window, scale, out, l_out, group):
    kf, vf = four.unpack(cache.k, cache.k_s, True) * cache.k_scale, four.unpack(cache.v, cache.v_s, False) * cache.v_scale
    dim = cache.head_dim
    for b, r in enumerate(vis):
        n = max(r)
        (kk, ok), (vv, _) = D.unpage(kf, cache.table, b, n), D.unpage(vf, cache.table, b, n)
        hi = torch.tensor(r, device="cuda").repeat_interleave(group)
        lo = (hi - window).clamp(min=0) if window else torch.zeros_like(hi)
        for h in range(cache.heads):
            mine = slice(h * group, (h + 1) * group)
            rows, kh, vh = q[b, :, mine].reshape(-1, dim).double(), kk[:, h].nan_to_num(0), vv[:, h].nan_to_num(0)
            o, l, A, mag = D.attention(rows, kh, vh, lo, hi, scale, ok)
            A = with_floor(A, rows, kh, vh, lo, hi, scale, ok, l, out.dtype)
            got_l = l_out[b, :, mine].reshape(-1) if l_out is not None else None
            D.check(out[b, :, mine].reshape(-1, dim), got_l, o, l, A, mag, n, dim, HF, f"request {b} head {h}")


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("qt", [BF, HF])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 255, 256, 257, 1000])
def test_decode_lengths(H, dim, qt, n):
    decode(H, 1, 1, 2, 4, dim, 16, qt, [[n]], seed=n, scales=(0.5, 1.5))


@pytest.mark.parametrize("qt", [BF, HF])
@pytest.mark.parametrize("dim,heads,group,nq,page", [
    (128, 1, 1, 1, 16), (128, 3, 7, 5, 48), (64, 5, 3, 8, 32), (128, 2, 16, 1, 64), (64, 1, 17, 1, 80), (128, 1, 32, 1, 16),
    (128, 1, 33, 1, 128), (64, 2, 16, 4, 64), (128, 1, 128, 8, 256), (64, 16, 1, 3, 16), (128, 2, 12, 2, 32), (64, 1, 25, 1, 16),
    (64, 3, 8, 8, 4096), (128, 1, 41, 3, 112)])
def test_decode_layouts(H, qt, dim, heads, group, nq, page):
    vis = [[max(0, e - nq + 1 + i) for i in range(nq)] for e in (700, 33, 5)]
    decode(H, 3, nq, heads, group, dim, page, qt, vis, seed=group * nq, spread=True)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 128, 5000])
def test_decode_window(H, window):
    """A sliding window; queries one apart, and queries far apart (gaps that none sees hold NaN)."""
    decode(H, 2, 3, 2, 4, 128, 32, BF, [[998, 999, 1000], [4, 5, 6]], window=window)
    decode(H, 1, 3, 1, 2, 64, 16, HF, [[40, 2000, 900]], window=window)
    decode(H, 1, 3, 2, 14, 128, 48, HF, [[40, 1200, 700]], window=window)


def test_decode_empty_requests(H):
    for group, nq in ((4, 2), (20, 2)):
        out = decode(H, 4, nq, 2, group, 128, 16, BF, [[0, 0], [0, 3], [100, 0], [0, 0]], max_vis=128)
        assert (out[0] == 0).all() and (out[1, 0] == 0).all() and (out[2, 1] == 0).all()


@pytest.mark.parametrize("group,nq", [(5, 5), (8, 1), (1, 1), (20, 3)])
@pytest.mark.parametrize("dim", [64, 128])
def test_decode_many_splits(H, group, nq, dim):
    decode(H, 1, nq, 1, group, dim, 64, BF, [[20001 + i for i in range(nq)]], seed=nq, scales=(0.5, 1.5))
    decode(H, 1, nq, 1, group, dim, 64, HF, [[900] * nq], seed=nq, max_vis=60000)


@pytest.mark.parametrize("dim,group,nq,page", [(128, 5, 5, 16), (64, 25, 1, 48), (64, 7, 1, 64), (128, 16, 8, 128), (128, 8, 1, 16)])
def test_decode_more_work_than_places(H, dim, group, nq, page):
    batch = 90
    vis = [[(37 * b * b + 11 * i) % 500 if b % 7 else 0 for i in range(nq)] for b in range(batch)]
    decode(H, batch, nq, 2, group, dim, page, HF, vis, seed=group, max_vis=520)


def test_decode_bad_pages_and_lengths_are_flagged(H):
    def edit(table):
        table[0, 3], table[1, 0] = -5, 1 << 30

    for group, nq in ((4, 1), (16, 3)):
        decode(H, 2, nq, 2, group, 128, 32, BF, [[400] * nq, [90] * nq], table_edit=edit, flags=H.HSA_FLAG_INDEX_RANGE)
    cache = cache_of(H, [64], 1, 64, 16, F4, 0)
    q = torch.randn(1, 1, 4, 64).to(BF).cuda()
    ws = H.new_paged_workspace(cache, 4, 1, 64)
    a, b = torch.empty_like(q), torch.empty_like(q)
    H.hsa_paged_attn_decode(cache, q, i32([[64]]), 64, 0.1, a, ws)
    clean(H)
    H.hsa_paged_attn_decode(cache, q, i32([[65]]), 64, 0.1, b, ws)
    clean(H, H.HSA_FLAG_INDEX_RANGE)
    assert torch.equal(a, b)


def test_decode_extreme_values(H):
    """Scales at both ends of E4M3, large and small queries and pool scales, and a NaN scale that a query sees."""
    for q_by, scales in ((1e-3, (2.0 ** -20, 2.0 ** 20)), (300.0, (2.0 ** -8, 1.0)), (1.0, (1.0, 2.0 ** -14))):
        for qt in (BF, HF):
            if qt is BF or scales[1] <= 1:               # values of 2^20 are past f16's range
                decode(H, 1, 1, 1, 8, 128, 16, qt, [[300]], q_by=q_by, scales=scales, spread=True)
    cache = cache_of(H, [300], 1, 128, 16, F4, 0)
    for ends in (1, 0x7E):
        cache.v_s.fill_(ends)
        q = torch.randn(1, 1, 8, 128).to(HF).cuda()
        out, ws = torch.empty_like(q), H.new_paged_workspace(cache, 8, 1, 300)
        H.hsa_paged_attn_decode(cache, q, i32([[300]]), 300, 0.1, out, ws)
        clean(H)
        check_decode(cache, q, [[300]], 0, 0.1, out, None, 8)
    cache.v_s[cache.table[0, 3].long(), 0, 5, 2] = 0x7F                  # position 53, dims 32 .. 47
    H.hsa_paged_attn_decode(cache, q, i32([[300]]), 300, 0.1, out, ws)
    clean(H)
    assert out[..., 32:48].isnan().all() and not out[..., :32].isnan().any() and not out[..., 48:].isnan().any()


def test_decode_long_cache_past_2_31_bytes(H):
    """Pools past 2^31 bytes: pages at both ends."""
    heads, dim, page = 16, 128, 64
    pages = (1 << 31) // (heads * page * dim // 2) + 40
    k, v = (torch.zeros(pages, heads, page, dim // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, heads, page, dim // 16), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ids = [pages - 1, 0, pages - 17, pages // 2, pages - 2]
    for p in ids:
        for pool, s, keys in ((k, ks, True), (v, vs, False)):
            pool[p], s[p] = four.pack(torch.randn(heads, page, dim, device="cuda"), keys)
    cache = H.PagedCache(k, v, i32([ids]), 1.0, 1.0, ks, vs)
    n = 5 * page - 7
    for group, nq in ((4, 1), (9, 3)):
        q = torch.randn(1, nq, heads * group, dim).to(BF).cuda()
        out = torch.empty_like(q)
        H.hsa_paged_attn_decode(cache, q, i32([[n] * nq]), n, 0.1, out, H.new_paged_workspace(cache, heads * group, nq, n))
        clean(H)
        kf, vf = (torch.cat([four.unpack(x[p], s[p], keys) for p in ids], 1) for x, s, keys in ((k, ks, True), (v, vs, False)))
        hi = torch.full((nq * group,), n, device="cuda")
        for h in range(heads):
            o, l, A, mag = D.attention(q[0, :, h * group:(h + 1) * group].reshape(-1, dim).double(), kf[h, :n], vf[h, :n], torch.zeros_like(hi), hi, 0.1)
            D.check(out[0, :, h * group:(h + 1) * group].reshape(-1, dim), None, o, l, A, mag, n, dim, HF, f"head {h}")
    rows = [torch.empty(n, heads, dim, dtype=BF, device="cuda") for _ in range(2)]
    H.hsa_paged_cache_read(cache, *rows)
    clean(H)
    assert torch.equal(rows[0], kf[:, :n].transpose(0, 1).to(BF)) and torch.equal(rows[1], vf[:, :n].transpose(0, 1).to(BF))


# --------------------------------------------------------------------------------------- verify
def fixed(x):
    """Probabilities in units of 2^-46, as exact whole numbers."""
    return (x.double().nan_to_num(0.0, posinf=1.0).clamp(0, 1) * 2.0 ** 46).round().long()


def verified(p, q, drafted, u_accept, u_sample, n):
    """(accepted, tokens, flags) of one request by the definition, in whole numbers."""
    nq, vocabulary = p.shape
    one = lambda x: min(max(float(x), 0.0), 1.0) if x == x else 0.0  # noqa: E731
    a, flags, without = 0, 0, None
    while a < n:
        x = int(drafted[a])
        if not 0 <= x < vocabulary:
            flags |= 1
            break
        if not float(u_accept[a]) * (one(q[a, x]) if q is not None else 1.0) < one(p[a, x]):
            without = x
            break
        a += 1
    w = fixed(p[a])
    if a < n and q is not None:
        # the comparison is of the entries themselves, the difference of their roundings
        w = (w - fixed(q[a])).clamp(min=0)
    elif a < n and without is not None:
        w = w.clone()
        w[without] = 0
    if not int(w.sum()):
        w = fixed(p[a])
    total = int(w.sum())
    y = -1
    if total:
        u = float(u_sample)
        u = 0.0 if u != u else min(max(u, 0.0), 1 - 2.0 ** -24)
        border = total * int(u * 2.0 ** 64) >> 64
        y = int((w.cumsum(0) <= border).sum())
    else:
        flags |= 8
    return a, [int(x) for x in drafted[:a]] + [y] + [-1] * (nq - 1 - a), flags


def verify(H, p, q, drafted, u_accept, u_sample, n=None):
    batch, nq, _ = p.shape
    accepted, tokens = torch.full((batch,), 77, dtype=torch.int32).cuda(), torch.full((batch, nq), 77, dtype=torch.int32).cuda()
    H.hsa_draft_verify(p, q, drafted, u_accept, u_sample, accepted, tokens, n_draft=n)
    counts = n.tolist() if n is not None else [nq - 1] * batch
    want_flags, got_a, got_t = 0, accepted.tolist(), tokens.tolist()
    for b in range(batch):
        if not 0 <= counts[b] < nq:
            want_flags |= counts[b] != -1
            assert got_a[b] == 77 and got_t[b] == [77] * nq
            continue
        a, t, f = verified(p[b].cpu(), None if q is None else q[b].cpu(), drafted[b].cpu(), u_accept[b].cpu(), u_sample[b].cpu(), counts[b])
        want_flags |= f
        assert (got_a[b], got_t[b]) == (a, t), f"request {b}"
    clean(H, want_flags)
    return got_a


def draft(batch, nq, n, dtype, seed, apart=0.7, by=2.5):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(batch, nq, n, generator=g) * by
    guess = logits[:, :-1] + apart * torch.randn(batch, nq - 1, n, generator=g)
    p, q = torch.softmax(logits, -1).to(dtype), torch.softmax(guess, -1).to(dtype)
    drafted = torch.multinomial(q.float().flatten(0, 1), 1, generator=g).view(batch, nq - 1) if nq > 1 else torch.empty(batch, 0)
    u = torch.rand(batch, nq - 1, generator=g), torch.rand(batch, generator=g)
    return p.cuda(), q.cuda(), drafted.to(torch.int32).cuda(), u[0].cuda(), u[1].cuda()


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("batch,nq,n", [(1, 1, 1), (1, 2, 2), (3, 5, 7), (1, 5, 131072), (7, 8, 4096), (40, 3, 50001), (5, 4, 4097), (400, 2, 1000), (2, 5, 127)])
def test_verify(H, dtype, batch, nq, n):
    p, q, drafted, ua, us = draft(batch, nq, n, dtype, seed=batch + n)
    kept = verify(H, p, q, drafted, ua, us)
    if batch >= 40:
        assert min(kept) == 0 and max(kept) == nq - 1                    # both ends are there
    verify(H, p, None, drafted, ua * 0.2, us)
    g = torch.Generator().manual_seed(n)
    verify(H, p, q, drafted, ua, us, torch.randint(-1, nq, (batch,), generator=g, dtype=torch.int32).cuda())


def test_verify_strides(H):
    """Rows at a distance (padded vocabularies), also where they do not start on 16-byte boundaries."""
    for n, room, off in ((1000, 1024, 0), (1000, 1001, 0), (999, 1003, 1), (50000, 50008, 8)):
        for dtype in (F32, BF):
            p, q, drafted, ua, us = draft(6, 4, n, dtype, seed=n)
            pp, qq = torch.full((6, 4, room + off), math.nan, dtype=dtype).cuda(), torch.full((6, 3, room + off), math.nan, dtype=dtype).cuda()
            pp[..., off:off + n], qq[..., off:off + n] = p, q
            verify(H, pp[..., off:off + n], qq[..., off:off + n], drafted, ua, us)


def test_verify_edges(H):
    """Randoms at their borders, weights at the ends, unequal and equal distributions, tokens out of range, rows without weight."""
    n = 3000
    p, q, drafted, ua, us = draft(12, 3, n, F32, seed=5)
    for value in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -3.0, 2.0 ** -40, math.nan, math.inf):
        verify(H, p, q, drafted, torch.full_like(ua, value), torch.full_like(us, value))
    for first in (0, n - 1, 1234):                                       # all weight at one place
        one = torch.zeros_like(p)
        one[..., first] = 1
        verify(H, one, q, drafted, ua, us)
        verify(H, one, None, drafted, ua, us)
    verify(H, p, p[:, :-1].contiguous(), drafted, ua, us)                # equal: everything stays
    verify(H, p, p[:, :-1].contiguous(), drafted, torch.ones_like(ua), us)   # u = 1 turns down, nothing is left of p: p itself
    bad = drafted.clone()
    bad[::2, 0], bad[1::3, 1] = -1, n
    verify(H, p, q, bad, ua, us)
    verify(H, p, None, bad, ua * 0.01, us)
    z = p.clone()
    z[3:6] = 0
    verify(H, z, q, drafted, ua, us)
    z[6, :, 100:200], z[7, :, 5], z[8] = math.nan, math.inf, -1.0
    verify(H, z, q, drafted, ua, us)
    verify(H, p, q, drafted, ua, us, i32([2, 1, 0, -1, 3, -2, 2, 2, 1, 0, -1, 9]))


def test_verify_follows_the_target(H):
    """Over many requests the first token's counts are those of p, whatever q is: chi squared below its mean + 8 deviations."""
    n, batch = 16, 20000
    g = torch.Generator().manual_seed(9)
    p1, q1 = torch.softmax(torch.randn(n, generator=g), -1), torch.softmax(torch.randn(n, generator=g), -1)
    drafted = torch.multinomial(q1, batch, replacement=True, generator=g).view(batch, 1).to(torch.int32).cuda()
    p, q = p1.cuda().expand(batch, 2, n).contiguous(), q1.cuda().expand(batch, 1, n).contiguous()
    ua, us = torch.rand(batch, 1, generator=g).cuda(), torch.rand(batch, generator=g).cuda()
    accepted, tokens = torch.empty(batch, dtype=torch.int32).cuda(), torch.empty(batch, 2, dtype=torch.int32).cuda()
    H.hsa_draft_verify(p, q, drafted, ua, us, accepted, tokens)
    clean(H)
    want = p1.double() * batch
    chi = ((torch.bincount(tokens[:, 0].long().cpu(), minlength=n) - want) ** 2 / want).sum().item()
    assert chi < (n - 1) + 8 * math.sqrt(2 * (n - 1))
    # E[accepted] = sum min(p, q)
    rate = torch.minimum(p1, q1).double().sum().item()
    assert abs(accepted.double().mean().item() - rate) < 6 * math.sqrt(rate * (1 - rate) / batch)


def test_verify_any_cut_gives_the_same_token(H):
    """A request alone (a cluster of CTAs) and among many (one CTA each): the same tokens."""
    p, q, drafted, ua, us = draft(310, 2, 5000, F32, seed=3)
    many = torch.empty(310, 2, dtype=torch.int32).cuda(), torch.empty(310, dtype=torch.int32).cuda()
    H.hsa_draft_verify(p, q, drafted, ua, us, many[1], many[0])
    t, a = torch.empty(1, 2, dtype=torch.int32).cuda(), torch.empty(1, dtype=torch.int32).cuda()
    for b in range(0, 310, 31):
        s = slice(b, b + 1)
        H.hsa_draft_verify(p[s], q[s], drafted[s], ua[s], us[s], a, t)
        assert torch.equal(t, many[0][s]) and torch.equal(a, many[1][s])
    clean(H)


# ------------------------------------------------------------------------------------- together
def step(H, s):
    """One speculative step of a dense layer over 4-bit pages: the draft's keys join the pages, its queries attend, the target's
    probabilities (a fixed projection of the outputs) verify it, and the lengths advance, all on the device."""
    H.hsa_paged_cache_append(s["cache"], s["k"], s["v"], s["inv"], q=s["q"], q_out=s["q_out"], start=s["start"])
    torch.add(s["start"][:, None], s["ahead"], out=s["vis64"])
    s["vis"].copy_(s["vis64"])
    H.hsa_paged_attn_decode(s["cache"], s["q_out"].view(s["out"].shape), s["vis"], s["most"], s["scale"], s["out"], s["ws"], lse=s["lse"])
    logits = s["out"].flatten(2).float() @ s["head"]
    torch.softmax(logits, -1, out=s["p"])
    H.hsa_draft_verify(s["p"], None, s["drafted"], s["ua"], s["us"], s["accepted"], s["tokens"])
    s["start"].add_(s["accepted"]).add_(1)


def new_step(H, seed, batch=5, nq=4, heads=2, group=5, dim=128, page=32, most=300):
    g = torch.Generator().manual_seed(seed)
    cache = cache_of(H, [most] * batch, heads, dim, page, F4, seed, (0.5, 0.75))
    rows = torch.randn(batch * nq, heads * (group + 2), dim, generator=g).to(BF).cuda()
    s = dict(cache=cache, most=most, scale=dim ** -0.5, inv=(10000.0 ** (-torch.arange(dim // 2) / (dim // 2))).float().cuda())
    s["q"], s["k"], s["v"] = rows.split((heads * group, heads, heads), 1)
    s["q_out"] = torch.empty(batch * nq, heads * group, dim, dtype=BF, device="cuda")
    s["start"] = torch.tensor([0, 17, 100, 250, 31][:batch]).cuda()
    s["ahead"] = torch.arange(1, nq + 1).cuda()[None]
    s["vis64"], s["vis"] = torch.zeros(batch, nq, dtype=torch.int64, device="cuda"), torch.zeros(batch, nq, dtype=torch.int32, device="cuda")
    s["out"] = torch.empty(batch, nq, heads * group, dim, dtype=BF, device="cuda")
    s["lse"] = torch.empty(batch, nq, heads * group, device="cuda")
    s["ws"] = H.new_paged_workspace(cache, heads * group, nq, most)
    s["head"] = torch.randn(heads * group * dim, 1000, generator=g).cuda() * 0.3
    s["p"] = torch.empty(batch, nq, 1000, device="cuda")
    s["drafted"] = torch.randint(0, 1000, (batch, nq - 1), generator=g, dtype=torch.int32).cuda()
    s["ua"], s["us"] = torch.rand(batch, nq - 1, generator=g).cuda() * 1e-3, torch.rand(batch, generator=g).cuda()
    s["accepted"], s["tokens"] = torch.empty(batch, dtype=torch.int32, device="cuda"), torch.empty(batch, nq, dtype=torch.int32, device="cuda")
    return s


def test_together(H):
    """The step's parts agree with each other and with the 64-bit forms: what was appended is what is read and attended to."""
    s = new_step(H, 1)
    cache, nq, batch = s["cache"], 4, 5
    old = s["start"].clone()
    step(H, s)
    clean(H)
    rows = [torch.empty(batch * nq, 2, 128, dtype=BF, device="cuda") for _ in range(2)]
    H.hsa_paged_cache_read(cache, *rows, start=old)
    clean(H)
    pos = (old[:, None] + torch.arange(nq).cuda()).flatten()
    want, _ = four.rotate(s["k"], pos, s["inv"], 0, True)
    scale = (want.unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True) / 6 * 1.125).expand(-1, -1, -1, 16).flatten(2)
    assert ((rows[0].double() - want).abs() <= scale * 1.01).all()       # half the largest step of the group's codes, 2 s
    vis = [[int(x) + i + 1 for i in range(nq)] for x in old]
    check_decode(cache, s["q_out"].view(s["out"].shape), vis, 0, s["scale"], s["out"], s["lse"], 5)
    for b in range(batch):
        a, t, _ = verified(s["p"][b].cpu(), None, s["drafted"][b].cpu(), s["ua"][b].cpu(), s["us"][b].cpu(), nq - 1)
        assert (int(s["accepted"][b]), s["tokens"][b].tolist()) == (a, t)
    assert torch.equal(s["start"], old + s["accepted"] + 1)


def test_chunk_behind_a_prefix_in_pages(H):
    """A chunk's attention over the rows that a read brings back, against 64 bits over the pages' own values."""
    heads, group, dim, past, new = 2, 4, 128, [100, 33], [40, 7]
    cache = cache_of(H, [140, 40], heads, dim, 16, F4, 3, (0.25, 0.5))
    x = torch.randn(47, heads * (group + 2), dim).to(HF).cuda()
    q, k, v = x.split((heads * group, heads, heads), 1)
    inv = (10000.0 ** (-torch.arange(64) / 64)).float().cuda()
    q_out, out = torch.empty(47, heads * group, dim, dtype=HF, device="cuda"), torch.empty(47, heads * group, dim, dtype=HF, device="cuda")
    H.hsa_paged_cache_append(cache, k, v, inv, q=q, q_out=q_out, cu=starts(new), start=torch.tensor(past).cuda())
    cu_k = starts([140, 40])
    kr, vr = (torch.empty(180, heads, dim, dtype=HF, device="cuda") for _ in range(2))
    H.hsa_paged_cache_read(cache, kr, vr, cu=cu_k)
    H.hsa_prompt_attn(q_out, kr, vr, starts(new), dim ** -0.5, out, cu_k=cu_k)
    clean(H)
    kf, vf = four.unpack(cache.k, cache.k_s, True) * 0.25, four.unpack(cache.v, cache.v_s, False) * 0.5
    t0 = 0
    for b, n in enumerate(new):
        (kk, _), (vv, _) = D.unpage(kf, cache.table, b, past[b] + n), D.unpage(vf, cache.table, b, past[b] + n)
        hi = torch.arange(past[b] + 1, past[b] + n + 1, device="cuda").repeat_interleave(group)
        for h in range(heads):
            rows = q_out[t0:t0 + n, h * group:(h + 1) * group].reshape(-1, dim)
            o, l, A, mag = D.attention(rows.double(), kk[:, h], vv[:, h], torch.zeros_like(hi), hi, dim ** -0.5)
            D.check(out[t0:t0 + n, h * group:(h + 1) * group].reshape(-1, dim), None, o, l, A, mag, past[b] + n, dim, HF, f"request {b} head {h}")
        t0 += n


KEYS = ("q_out", "out", "lse", "accepted", "tokens", "start")


def test_captured_and_on_another_stream(H):
    """Three steps captured as one graph and replayed, and on a side stream, give the bits of eager steps."""
    s = new_step(H, 2)
    for _ in range(3):
        step(H, s)
    want = [s[x].clone() for x in KEYS] + copies(s["cache"])
    for mode in ("stream", "graph"):
        s = new_step(H, 2)
        first = s["start"].clone()
        pages = copies(s["cache"])
        torch.cuda.synchronize()
        if mode == "stream":
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3):
                    step(H, s)
            torch.cuda.synchronize()
        else:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                step(H, s)               # libraries that allocate do so before the capture
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(H, s)
            for _ in range(2):
                s["start"].copy_(first)
                for t, old in zip((s["cache"].k, s["cache"].v, s["cache"].k_s, s["cache"].v_s), pages):
                    t.copy_(old)
                for _ in range(3):
                    graph.replay()
            torch.cuda.synchronize()
        for name, a, b in zip(KEYS + ("k", "v", "k_s", "v_s"), [s[x] for x in KEYS] + copies(s["cache"]), want):
            assert torch.equal(a, b), (mode, name)
    clean(H)


def test_steps_at_the_same_time(H):
    """Steps of different caches on three streams at once give the bits of steps one by one."""
    want = []
    for seed in range(3):
        s = new_step(H, seed)
        for _ in range(4):
            step(H, s)
        want.append([s[x].clone() for x in KEYS])
    states = [new_step(H, seed) for seed in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(4):
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                step(H, s)
    torch.cuda.synchronize()
    for s, w in zip(states, want):
        assert all(torch.equal(s[x], y) for x, y in zip(KEYS, w))
    clean(H)
