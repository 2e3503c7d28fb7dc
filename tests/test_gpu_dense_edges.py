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
