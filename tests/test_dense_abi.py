"""Refusals of the dense attention calls that return before any CUDA call (no GPU needed), on made-up
addresses that nothing reads, and the argument checks of their Python binding."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def H():
    from hierarchical_sparse_attention_index_gb300 import build
    try:
        build.nvcc()
    except RuntimeError as e:
        pytest.skip(str(e))
    build.build()
    import hierarchical_sparse_attention_index_gb300 as h
    h.load_library()
    return h


INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


def cache(H, **change):
    f = dict(batch=2, heads=4, head_dim=128, page_size=16, dtype=H.HSA_BF16, flags=0, n_pages=100, max_pages=64, k=0x1000,
             v=0x2000, table=0x3000, k_scale=1.0, v_scale=1.0)
    f.update(change)
    return H.hsa_paged_cache(*f.values())


BAD_CACHES = [
    (dict(batch=0), SHAPE), (dict(heads=0), SHAPE), (dict(heads=1025), SHAPE), (dict(head_dim=96), SHAPE), (dict(page_size=8), SHAPE),
    (dict(page_size=24), SHAPE), (dict(page_size=4112), SHAPE), (dict(n_pages=0), SHAPE), (dict(n_pages=1 << 31), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(max_pages=(1 << 31) // 16), SHAPE), (dict(dtype=3), INVALID), (dict(flags=1), INVALID),
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(table=0), INVALID), (dict(k_scale=0.0), INVALID),
    (dict(dtype=2, v_scale=-1.0), INVALID), (dict(dtype=2, k_scale=NAN), INVALID), (dict(dtype=2, k_scale=INF), INVALID),
    (dict(k_scale=2.0), INVALID), (dict(k=0x1008), ALIGN), (dict(v=0x2001), ALIGN)]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_bad_caches(H, change, code):
    lib, c = H.load_library(), cache(H, **change)
    r = ctypes.byref(c)
    assert lib.hsa_paged_cache_write(r, 0x10, 0x20, H.HSA_BF16, 512, 512, 4, 0x30, 0x40, None) == code
    assert lib.hsa_paged_attn_decode(r, 0x10, H.HSA_BF16, 8, 0x20, 1, 64, 0, 0.1, 0x30, 0x40, 0x50, 1 << 30, None) == code


def test_write_refusals(H):
    lib, c = H.load_library(), cache(H)
    ok = dict(k=0x10, v=0x20, dtype=H.HSA_BF16, k_stride=512, v_stride=512, n=4, cu=0x30, start=0x40)

    def call(c=c, **change):
        return lib.hsa_paged_cache_write(ctypes.byref(c) if c is not None else None, *{**ok, **change}.values(), None)

    assert call(c=None) == INVALID
    assert call(k=None) == INVALID and call(v=None) == INVALID
    assert call(dtype=H.HSA_F16) == INVALID and call(dtype=H.HSA_E4M3) == INVALID and call(dtype=-1) == INVALID
    assert call(c=cache(H, dtype=H.HSA_E4M3), dtype=H.HSA_E4M3) == INVALID
    assert call(n=-1) == SHAPE and call(n=1 << 31) == SHAPE
    assert call(k_stride=504) == SHAPE and call(v_stride=516) == SHAPE and call(k_stride=1 << 31) == SHAPE
    assert call(cu=None, n=3) == SHAPE                  # does not divide over the requests
    assert call(k=0x18) == ALIGN and call(v=0x21) == ALIGN
    assert call(n=0, k=None, v=None) == 0               # nothing to write: no launch


def test_decode_refusals(H):
    lib, c = H.load_library(), cache(H)
    ok = dict(q=0x10, dtype=H.HSA_BF16, heads_q=8, vis=0x20, nq=2, max_vis=1000, window=0, scale=0.1, out=0x30, lse=0x40, ws=0x50,
              ws_bytes=1 << 30)

    def call(c=c, **change):
        return lib.hsa_paged_attn_decode(ctypes.byref(c) if c is not None else None, *{**ok, **change}.values(), None)

    assert call(c=None) == INVALID
    for name in ("q", "vis", "out"):
        assert call(**{name: None}) == INVALID
    assert call(dtype=H.HSA_F16) == INVALID and call(dtype=H.HSA_E4M3) == INVALID
    assert call(c=cache(H, dtype=H.HSA_E4M3), dtype=H.HSA_E4M3) == INVALID
    for scale in (0.0, -1.0, NAN, INF):
        assert call(scale=scale) == INVALID
    assert call(window=-1) == INVALID
    assert call(heads_q=0) == SHAPE and call(heads_q=10) == SHAPE and call(heads_q=4 * 129) == SHAPE
    assert call(nq=0) == SHAPE and call(nq=9) == SHAPE
    assert call(max_vis=-1) == SHAPE and call(max_vis=64 * 16 + 1) == SHAPE
    assert call(c=cache(H, max_pages=1 << 20), max_vis=(1 << 20) + 1) == SHAPE
    assert call(q=0x11) == ALIGN and call(out=0x38) == ALIGN and call(ws=0x58) == ALIGN
    need = lib.hsa_paged_attn_workspace_bytes(ctypes.byref(c), 8, 2, 1000)
    assert call(ws=None) == WORKSPACE and call(ws_bytes=need - 1) == WORKSPACE and call(ws_bytes=0) == WORKSPACE


def test_workspace_bytes(H):
    lib = H.load_library()

    def need(heads_q=8, nq=2, max_vis=1000, **change):
        return lib.hsa_paged_attn_workspace_bytes(ctypes.byref(cache(H, **change)), heads_q, nq, max_vis)

    assert lib.hsa_paged_attn_workspace_bytes(None, 8, 2, 1000) == 0
    assert need() > 0 and need(max_vis=0) > 0
    assert need(heads_q=9) == 0 and need(nq=9) == 0 and need(max_vis=1025) == 0 and need(head_dim=32) == 0
    assert need(k=0, v=0, table=0) == need()            # the pointers are not looked at
    sizes = [need(max_vis=m, max_pages=1 << 16) for m in range(0, 1 << 20, 4099)]
    assert sizes == sorted(sizes)                       # a workspace for a bound serves every smaller one


def test_prompt_refusals(H):
    lib = H.load_library()
    ok = dict(batch=2, heads_q=8, heads_kv=4, head_dim=128, dtype=H.HSA_BF16, window=0, n_q=100, n_k=100, q=0x10, k=0x20, v=0x30,
              q_stride=1024, k_stride=512, v_stride=512, out_stride=1024, cu_q=0x44, cu_k=None, sm_scale=0.1, out=0x50,
              lse=None)

    def call(**change):
        return lib.hsa_prompt_attn(ctypes.byref(H.hsa_prompt_args(*{**ok, **change}.values())), None)

    assert lib.hsa_prompt_attn(None, None) == INVALID
    assert call(dtype=H.HSA_E4M3) == INVALID and call(dtype=9) == INVALID and call(window=-1) == INVALID
    for scale in (0.0, -0.5, NAN, INF):
        assert call(sm_scale=scale) == INVALID
    for name in ("q", "k", "v", "out", "cu_q"):
        assert call(**{name: None}) == INVALID
    assert call(batch=0) == SHAPE and call(heads_kv=0) == SHAPE and call(head_dim=256) == SHAPE
    assert call(heads_kv=1025, heads_q=1025, q_stride=1 << 18) == SHAPE
    assert call(heads_q=6) == SHAPE and call(heads_q=0) == SHAPE and call(heads_q=4 * 132, q_stride=1 << 17) == SHAPE
    assert call(n_q=-1) == SHAPE and call(n_k=-1) == SHAPE and call(n_q=1 << 31) == SHAPE and call(n_k=1 << 31) == SHAPE
    for name, short in (("q_stride", 1016), ("out_stride", 1016), ("k_stride", 504), ("v_stride", 504)):
        assert call(**{name: short}) == SHAPE and call(**{name: 1028}) == SHAPE and call(**{name: 1 << 31}) == SHAPE
    for name in ("q", "k", "v", "out"):
        assert call(**{name: 0x1008}) == ALIGN
    assert call(n_q=0, q=None, out=None, cu_q=None) == 0     # no queries: no launch


def test_binding_checks(H):
    """The binding takes addresses of tensors, so it refuses what their addresses cannot stand for."""
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 4, dtype=torch.int32)
    for bad in (dict(table=table.long()), dict(v=k.half()), dict(v=k[:2]), dict(k=k.transpose(1, 2), v=k.transpose(1, 2)),
                dict(k=k.float(), v=k.float()), dict(table=table[0]), dict(k=k[0], v=k[0])):
        with pytest.raises(ValueError):
            H.PagedCache(**{**dict(k=k, v=k.clone(), table=table), **bad})
    c = H.PagedCache(k, k.clone(), table)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    # CPU tensors never reach the library
    with pytest.raises(ValueError):
        H.hsa_paged_cache_write(c, x, x)
    with pytest.raises(ValueError):
        H.hsa_paged_attn_decode(c, x[None], torch.zeros(1, 3, dtype=torch.int32), 3, 0.1, x[None], None)
    with pytest.raises(ValueError):
        H.hsa_prompt_attn(x, x, x, torch.zeros(2, dtype=torch.int32), 0.1, x)
    # strides that the library has no argument for
    for t in (x.transpose(1, 2), torch.zeros(3, 4, 64, dtype=torch.bfloat16)[:, ::2], x[..., :32], x[0]):
        with pytest.raises(ValueError):
            H._rows("x", t, 2, 64)
    assert H._rows("x", torch.zeros(3, 6, 64)[:, 1:3], 2, 64) == 6 * 64
    assert H._rows("x", torch.zeros(1, 2, 64), 2, 64) == 128


def test_grids_that_are_too_large(H):
    """Sizes that are each in range but whose grid is not are refused, not left to a failing launch."""
    lib = H.load_library()
    wide = dict(batch=1, heads_q=131072, heads_kv=1024, head_dim=64, dtype=H.HSA_BF16, window=0, n_q=1 << 27, n_k=100, q=0x10,
                k=0x20, v=0x30, q_stride=1 << 23, k_stride=1 << 16, v_stride=1 << 16, out_stride=1 << 23, cu_q=0x44, cu_k=None,
                sm_scale=0.1, out=0x50, lse=None)
    for change in (dict(), dict(n_q=100, batch=(1 << 20) + 1)):
        assert lib.hsa_prompt_attn(ctypes.byref(H.hsa_prompt_args(*{**wide, **change}.values())), None) == SHAPE
    c = cache(H, batch=1 << 20, heads=1024)
    assert lib.hsa_paged_attn_decode(ctypes.byref(c), 0x10, H.HSA_BF16, 1 << 17, 0x40, 1, 1024, 0, 0.1, 0x10, None, 0x100, 1 << 62,
                                     None) == SHAPE


@pytest.mark.parametrize("nq,group,dtype", [(5, 7, "HSA_BF16"), (1, 8, "HSA_BF16"), (5, 7, "HSA_E4M3")])
def test_workspace_holds_for_shorter_lengths(H, nq, group, dtype):
    """A workspace for max_vis serves every smaller one."""
    lib = H.load_library()
    for batch in (1, 3, 16, 64, 200):
        c = cache(H, batch=batch, dtype=getattr(H, dtype), max_pages=10000)
        sizes = [lib.hsa_paged_attn_workspace_bytes(ctypes.byref(c), 4 * group, nq, n) for n in range(0, 160000, 61)]
        assert min(sizes) > 0 and sizes == sorted(sizes)
