"""Borders of what the calls of a speculative step promise: angles of turning back and of positions far past any page."""
import math

import pytest
import torch

from tests import four
from tests import test_gpu_step as S
from tests.test_gpu_step import HF, H  # noqa: F401  (H is a fixture)

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
