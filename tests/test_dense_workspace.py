"""The workspace of hsa_paged_attn_decode serves every shorter length and every window (CPU only: the calls
are refused for a workspace address that is not aligned, which is looked at after its size)."""
import ctypes

import pytest

from tests.test_dense_abi import ALIGN, H, cache  # noqa: F401  (H is a fixture)


@pytest.mark.parametrize("dtype,nq,group", [("HSA_E4M3", 5, 7), ("HSA_E4M3", 8, 16), ("HSA_E4M3", 1, 20), ("HSA_BF16", 3, 8),
                                            ("HSA_BF16", 1, 17), ("HSA_BF16", 1, 4), ("HSA_F16", 5, 7), ("HSA_F16", 8, 42)])
def test_workspace_serves_shorter_lengths_and_windows(H, dtype, nq, group):  # noqa: F811
    lib = H.load_library()
    code = getattr(H, dtype)
    q_type = H.HSA_BF16 if code == H.HSA_E4M3 else code
    for batch in (1, 3, 8, 17, 40, 64, 150, 700):
        c = cache(H, batch=batch, dtype=code, max_pages=1 << 14)
        r = ctypes.byref(c)
        for most in (64, 1000, 4097, 30000, 200000):
            need = lib.hsa_paged_attn_workspace_bytes(r, 4 * group, nq, most)
            for n in {0, 1, most // 7, most // 3, most // 2, most * 3 // 4, most - 1, most}:
                for window in (0, 1, 100, most // 2, most):
                    got = lib.hsa_paged_attn_decode(r, 0x10, q_type, 4 * group, 0x20, nq, n, window, 0.1, 0x30, None, 0x48, need, None)
                    assert got == ALIGN, (batch, most, n, window)
