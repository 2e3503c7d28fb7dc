"""Borders of what the calls of a speculative step promise: angles of turning back and of positions far past any page, randoms
whose product with a sum is a few of its units, every place written for rows that are no distributions, and the largest vocabularies."""
import math

import pytest
import torch

from tests import four
from tests import test_gpu_step as S
from tests.test_gpu_step import BF, HF, H  # noqa: F401  (H is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("halves", [True, False])
@pytest.mark.parametrize("first", [0, 123456789, (1 << 31) - 4096, 1 << 40, 1 << 44])
def test_append_angles_of_either_sign(H, first, halves):  # noqa: F811
    """Rotated queries at positions without a place, for pairs that turn forth and back by the same frequencies. The angle is off by
    2^-52 of pos inv_freq / 2 pi turns and by |pos| 2^-64 turns at most; the 64-bit form's own product by 2^-53 of itself. The rest
    as in tests/test_gpu_step.py: 2^-21 (|x| + |y|) in fp32, then half a step of the 16-bit result."""
    slow = torch.tensor([1e-4, 1e-7, 3e-3, 2.0 ** -20, 160000.0 ** (-126 / 128), 7e-6, 2.0 ** -30, 5e-4] * 2)
    inv = torch.cat((slow, -slow)).float().cuda()
    g = torch.Generator().manual_seed(first % 1000)
    n, dim = 40, 64
    x = torch.randn(n, 1, dim, generator=g).to(HF).cuda()
    cache, out = S.cache_of(H, [16], 1, dim, 16, HF, 0), torch.empty_like(x)
    H.hsa_paged_cache_append(cache, x, x, inv, q=x, q_out=out, start=torch.tensor([first]).cuda(),
                             pairs=H.HSA_ROPE_HALVES if halves else H.HSA_ROPE_NEIGHBOURS)
    S.clean(H, H.HSA_FLAG_WRITE_RANGE)
    pos = torch.arange(first, first + n, device="cuda")
    want, size = four.rotate(x, pos, inv, 0, halves)
    each = torch.cat((inv, inv)) if halves else inv.repeat_interleave(2)
    angle = pos.double()[:, None] * (1.5 * 2.0 ** -52 * each.double().abs() + 2 * math.pi * 2.0 ** -64)
    bound = 2.0 ** -11 * want.abs() + (2.0 ** -21 + angle[:, None]) * size * 1.001 + 2.0 ** -25
    off = (out.double() - want).abs()
    assert (off <= bound).all(), f"{(off / bound).max()} times the bound"


@pytest.mark.parametrize("low", [1, 2, 3, 7, 50])
@pytest.mark.parametrize("dtype", [torch.float32, BF, HF])
def test_verify_small_randoms(H, dtype, low):  # noqa: F811
    """A random so small that its product with the sum is a few units: the first token holds `low` of them. At the smallest random
    whose product reaches `low` the token is the next one, at any below it the first."""
    n, at = 2000, (700, 1500, 1999)
    unit = 2.0 ** -46 if dtype is not HF else 2.0 ** -24                 # (f16 has no smaller value)
    p = torch.zeros(1, 1, n)
    p[0, 0, at[0]], p[0, 0, at[1]], p[0, 0, at[2]] = low * unit, 0.3, 0.4
    p = p.to(dtype).cuda()
    w = S.fixed(p[0, 0]).tolist()
    total, first = sum(w), w[at[0]]
    shift = 0                                                            # u = m 2^-shift, m of 24 bits
    while -(-(first << shift) // total) < 1 << 23:
        shift += 1
    m = -(-(first << shift) // total)                                    # total m 2^-shift >= first, for the first time
    assert m < 1 << 24
    cases = [m - 1, m, m + 1, m - 2 if m - 2 >= 1 << 23 else m]
    u = torch.tensor([c * 2.0 ** -shift for c in cases], dtype=torch.float64).float().cuda()
    assert [int(x * 2 ** shift) for x in u.double().tolist()] == cases
    k = len(cases)
    accepted, tokens = torch.full((k,), 77, dtype=torch.int32).cuda(), torch.full((k, 1), 77, dtype=torch.int32).cuda()
    H.hsa_draft_verify(p.expand(k, 1, n).contiguous(), None, torch.empty(k, 0, dtype=torch.int32, device="cuda"),
                       torch.empty(k, 0, device="cuda"), u, accepted, tokens)
    S.clean(H)
    want = [at[0] if total * c < first << shift else at[1] for c in cases]
    assert tokens[:, 0].tolist() == want and accepted.tolist() == [0] * k


def test_verify_of_garbage_writes_every_place(H):  # noqa: F811
    """Rows that are no distributions (too large a sum, random bits): each request gets its kept tokens, one of the vocabulary behind
    them, and -1 in the rest; nothing is left as it was, and nothing else is written."""
    batch, nq, n, was = 40, 4, 5003, -77
    g = torch.Generator().manual_seed(1)
    for p in (torch.ones(batch, nq, n), torch.randint(-2 ** 31, 2 ** 31 - 1, (batch, nq, n), generator=g, dtype=torch.int32).view(torch.float32)):
        p = p.cuda()
        q = p[:, 1:].contiguous().flip(1)
        drafted = torch.randint(0, n, (batch, nq - 1), generator=g, dtype=torch.int32).cuda()
        room = torch.full((batch * nq + 32,), was, dtype=torch.int32, device="cuda")
        tokens, accepted = room[16:16 + batch * nq].view(batch, nq), torch.full((batch,), was, dtype=torch.int32, device="cuda")
        for ua in (torch.rand(batch, nq - 1, generator=g), torch.zeros(batch, nq - 1), torch.full((batch, nq - 1), 2.0)):
            tokens.fill_(was)
            accepted.fill_(was)
            H.hsa_draft_verify(p, q, drafted, ua.cuda(), torch.rand(batch, generator=g).cuda(), accepted, tokens)
            S.clean(H)
            assert ((accepted >= 0) & (accepted < nq)).all()
            assert (room[:16] == was).all() and (room[16 + batch * nq:] == was).all()
            place, a = torch.arange(nq).cuda()[None], accepted[:, None]
            y = tokens.gather(1, a.long())
            assert ((y >= 0) & (y < n)).all()
            want = torch.where(place < a, torch.cat((drafted, drafted[:, :1]), 1), torch.where(place == a, y, -1))
            assert torch.equal(tokens, want)


@pytest.mark.parametrize("dtype,n", [(torch.float32, 1 << 24), (torch.float32, (1 << 24) - 1), (BF, 1 << 24), (HF, (1 << 24) - 129)])
def test_verify_largest_vocabularies(H, dtype, n):  # noqa: F811
    """As many entries as a row may have, and odd numbers near it: draws at both ends of the row and between."""
    p, q, drafted, ua, _ = S.draft(3, 2, n, dtype, seed=3)
    for at in (0.0, 0.5, 1.0 - 2.0 ** -24):
        us = torch.full((3,), at, device="cuda")
        S.verify(H, p, q, drafted, torch.tensor([[0.0], [2.0], [0.9]], device="cuda"), us)
        S.verify(H, p, None, drafted, ua, us)
