"""Refusals of the calls of a speculative step over a paged cache (rotated append, read, 4-bit pages, verification of a draft)
that return before any CUDA call (no GPU needed), on made-up addresses that nothing reads, and the checks of their binding."""
import ctypes

import pytest
import torch

from tests import four
from tests.test_dense_abi import ALIGN, BAD_CACHES, INVALID, SHAPE, WORKSPACE, H, cache  # noqa: F401  (H is a fixture)


def four_bits(H, **change):  # noqa: F811
    return cache(H, **{**dict(dtype=H.HSA_E2M1), **change, **dict(k_s=change.get("k_s", 0x4000), v_s=change.get("v_s", 0x5000))})


def append_call(H, c=None, **change):  # noqa: F811
    ok = dict(dtype=H.HSA_BF16, heads_q=8, rotary_at=0, rotary_dims=128, pairs=0, n_tokens=4, q=0x10, k=0x20, v=0x30, q_stride=1024,
              k_stride=512, v_stride=512, out_stride=1024, cu=0x44, start=0x48, inv_freq=0x54, q_out=0x60)
    c = cache(H) if c is None else c
    return H.load_library().hsa_paged_cache_append(ctypes.byref(c), ctypes.byref(H.hsa_append_args(*{**ok, **change}.values())), None)


def test_four_bit_caches(H):  # noqa: F811
    lib = H.load_library()

    def calls(c):
        r = ctypes.byref(c)
        return {lib.hsa_paged_cache_write(r, 0x10, 0x20, H.HSA_BF16, 512, 512, 4, 0x30, 0x40, None),
                lib.hsa_paged_cache_read(r, 0x10, 0x20, H.HSA_BF16, 512, 512, 4, 0x30, 0x40, None), append_call(H, c),
                lib.hsa_paged_attn_decode(r, 0x10, H.HSA_BF16, 8, 0x20, 1, 64, 0, 0.1, 0x30, 0x40, 0x50, 1 << 30, None)}

    assert calls(four_bits(H, k_s=0)) == {INVALID} and calls(four_bits(H, v_s=0)) == {INVALID}
    assert calls(four_bits(H, k_s=0x4008)) == {ALIGN} and calls(four_bits(H, v_s=0x5001)) == {ALIGN}
    assert calls(four_bits(H, k_scale=0.0)) == {INVALID} and calls(four_bits(H, head_dim=32)) == {SHAPE}
    assert calls(cache(H, dtype=4)) == {INVALID}                     # probabilities only
    # types that a 4-bit cache takes, and a workspace that serves it
    c = four_bits(H, k_scale=0.5, v_scale=2.0, max_pages=1 << 12)
    r = ctypes.byref(c)
    for dtype in (H.HSA_E4M3, H.HSA_E2M1, H.HSA_F32):
        assert lib.hsa_paged_cache_read(r, 0x10, 0x20, dtype, 512, 512, 4, 0x30, 0x40, None) == INVALID
        assert lib.hsa_paged_attn_decode(r, 0x10, dtype, 8, 0x20, 1, 64, 0, 0.1, 0x30, 0x40, 0x50, 1 << 30, None) == INVALID
    for group, nq in ((1, 1), (8, 1), (7, 5), (16, 8), (128, 8)):
        for most in (64, 4097, 60000):
            need = lib.hsa_paged_attn_workspace_bytes(r, 4 * group, nq, most)
            assert need > 0
            for n in {0, 1, most // 3, most - 1, most}:
                for window in (0, 1, 100, most):
                    got = lib.hsa_paged_attn_decode(r, 0x10, H.HSA_BF16, 4 * group, 0x20, nq, n, window, 0.1, 0x30, None, 0x48, need, None)
                    assert got == ALIGN, (group, nq, most, n, window)
            assert lib.hsa_paged_attn_decode(r, 0x10, H.HSA_F16, 4 * group, 0x20, nq, most, 0, 0.1, 0x30, None, 0x50, 0, None) == WORKSPACE


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_bad_caches(H, change, code):  # noqa: F811
    c = cache(H, **change)
    assert append_call(H, c) == code
    assert H.load_library().hsa_paged_cache_read(ctypes.byref(c), 0x10, 0x20, H.HSA_BF16, 512, 512, 4, 0x30, 0x40, None) == code


def test_append_refusals(H):  # noqa: F811
    lib, c = H.load_library(), cache(H)
    assert lib.hsa_paged_cache_append(ctypes.byref(c), None, None) == INVALID
    assert lib.hsa_paged_cache_append(None, ctypes.byref(H.hsa_append_args()), None) == INVALID
    for name in ("k", "v", "q", "q_out", "inv_freq"):
        assert append_call(H, **{name: None}) == INVALID
    assert append_call(H, dtype=H.HSA_F16) == INVALID and append_call(H, dtype=H.HSA_E4M3) == INVALID
    assert append_call(H, pairs=2) == INVALID and append_call(H, pairs=-1) == INVALID
    assert append_call(H, n_tokens=-1) == SHAPE and append_call(H, n_tokens=1 << 31) == SHAPE
    assert append_call(H, heads_q=-1) == SHAPE and append_call(H, heads_q=131073) == SHAPE
    for at, dims in ((8, 64), (-16, 64), (0, 48), (0, -32), (0, 160), (16, 128), (144, 0), (64, 96)):
        assert append_call(H, rotary_at=at, rotary_dims=dims) == SHAPE
    for name in ("q_stride", "k_stride", "v_stride", "out_stride"):
        assert append_call(H, **{name: 504}) == SHAPE and append_call(H, **{name: 1028}) == SHAPE
        assert append_call(H, **{name: 1 << 31}) == SHAPE
    assert append_call(H, cu=None, n_tokens=3) == SHAPE
    for name in ("q", "k", "v", "q_out"):
        assert append_call(H, **{name: 0x1008}) == ALIGN
    assert append_call(H, n_tokens=0, q=None, k=None, v=None, q_out=None, inv_freq=None) == 0     # nothing to append: no launch


def test_read_refusals(H):  # noqa: F811
    lib, c = H.load_library(), cache(H)
    ok = dict(k=0x10, v=0x20, dtype=H.HSA_BF16, k_stride=512, v_stride=512, n=4, cu=0x30, start=0x40)

    def call(c=c, **change):
        return lib.hsa_paged_cache_read(ctypes.byref(c) if c is not None else None, *{**ok, **change}.values(), None)

    assert call(c=None) == INVALID and call(k=None) == INVALID and call(v=None) == INVALID
    assert call(dtype=H.HSA_F16) == INVALID and call(dtype=H.HSA_E2M1) == INVALID
    assert call(n=-1) == SHAPE and call(n=1 << 31) == SHAPE and call(cu=None, n=3) == SHAPE
    assert call(k_stride=504) == SHAPE and call(v_stride=516) == SHAPE and call(k_stride=1 << 31) == SHAPE
    assert call(k=0x18) == ALIGN and call(v=0x21) == ALIGN
    assert call(n=0, k=None, v=None) == 0


def test_verify_refusals(H):  # noqa: F811
    lib = H.load_library()
    ok = dict(batch=2, nq=5, vocabulary=1000, dtype=H.HSA_F32, p=0x10, q=0x20, p_stride=1000, q_stride=1000, drafted=0x30, n_draft=0x34,
              u_accept=0x38, u_sample=0x3C, accepted=0x40, tokens=0x44)

    def call(**change):
        return lib.hsa_draft_verify(ctypes.byref(H.hsa_verify_args(*{**ok, **change}.values())), None)

    assert lib.hsa_draft_verify(None, None) == INVALID
    for name in ("p", "drafted", "u_accept", "u_sample", "accepted", "tokens"):
        assert call(**{name: None}) == INVALID
    for dtype in (H.HSA_E4M3, H.HSA_E2M1, -1, 5):
        assert call(dtype=dtype) == INVALID
    assert call(batch=0) == SHAPE and call(batch=(1 << 20) + 1) == SHAPE and call(nq=0) == SHAPE and call(nq=9) == SHAPE
    assert call(vocabulary=0) == SHAPE and call(vocabulary=(1 << 24) + 1, p_stride=1 << 25, q_stride=1 << 25) == SHAPE
    assert call(p_stride=999) == SHAPE and call(q_stride=999) == SHAPE and call(p_stride=1 << 31) == SHAPE and call(q_stride=1 << 31) == SHAPE
    assert call(p=0x12) == ALIGN and call(q=0x11) == ALIGN and call(dtype=H.HSA_BF16, p=0x11) == ALIGN
    for name in ("drafted", "n_draft", "u_accept", "u_sample", "accepted", "tokens"):
        assert call(**{name: 0x1002}) == ALIGN


def test_binding_checks(H):  # noqa: F811
    """The binding takes addresses of tensors, so it refuses what their addresses cannot stand for."""
    k, s = torch.zeros(4, 2, 16, 32, dtype=torch.uint8), torch.zeros(4, 2, 16, 4, dtype=torch.float8_e4m3fn)
    table = torch.zeros(1, 4, dtype=torch.int32)
    good = dict(k=k, v=k.clone(), table=table, k_s=s, v_s=s.clone())
    for bad in (dict(k_s=None), dict(v_s=None), dict(k_s=s[:2]), dict(v_s=s.float()), dict(k_s=s.transpose(1, 2)), dict(v=k.bfloat16()),
                dict(k=k.bfloat16(), v=k.bfloat16())):
        with pytest.raises(ValueError):
            H.PagedCache(**{**good, **bad})
    c = H.PagedCache(**good)
    assert (c.head_dim, c.dtype) == (64, H.HSA_E2M1)
    H.PagedCache(**{**good, **dict(k_s=s.view(torch.uint8), v_s=s.view(torch.uint8))})
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    f = torch.zeros(32)
    # CPU tensors never reach the library
    for call in (lambda: H.hsa_paged_cache_append(c, x, x, f), lambda: H.hsa_paged_cache_read(c, x, x),
                 lambda: H.hsa_draft_verify(torch.zeros(1, 1, 5), None, torch.zeros(1, 0, dtype=torch.int32), torch.zeros(1, 0),
                                            torch.zeros(1), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()
    # rows of probabilities that the library has no stride for
    p = torch.zeros(3, 4, 10)
    assert H._probabilities("p", p, (3, 4, 10)) == 10 and H._probabilities("p", torch.zeros(3, 4, 16)[..., :10], (3, 4, 10)) == 16
    assert H._probabilities("p", torch.zeros(3, 8, 10)[:, ::2], (3, 4, 10)) == 20 and H._probabilities("p", p[:, 1:2], (3, 1, 10)) == 40
    for t in (torch.zeros(3, 8, 10)[:, :4], p.transpose(1, 2).contiguous().transpose(1, 2), p[:2], torch.zeros(3, 4, 20)[..., ::2]):
        with pytest.raises(ValueError):
            H._probabilities("p", t, (3, 4, 10))


def test_plain_forms():
    """The tests' own forms of 4-bit rows: packing and unpacking give the nearest values, in both byte orders."""
    x = torch.randn(5, 128, generator=torch.Generator().manual_seed(1)).double()
    for keys in (True, False):
        for dim in (64, 128):
            assert sorted(four.order(dim, keys).tolist()) == list(range(dim // 2))
            b, s = four.pack(x[:, :dim], keys)
            y = four.unpack(b, s, keys)
            scale = four.SCALES[s.long() - 1].repeat_interleave(16, -1)
            assert ((y - x[:, :dim]).abs() <= scale).all() and (x[:, :dim].abs() <= 6 * scale).all()
            four.check_group(b, s, x[:, :dim], torch.zeros_like(x[:, :dim]), keys)
    assert four.scale_of(torch.tensor([0.0, 6 * 2.0 ** -9, 6 * 2.0 ** -9 + 1e-9, 6.0, 1e9])).tolist() == [1, 1, 2, 0x38, 0x7E]
    assert four.code_of(torch.tensor([0.25, 0.75, 2.5, -3.5, 5.0, 5.1, -9.0])).tolist() == [0, 2, 4, -6, 6, 7, -7]


def test_records_as_bytes(H):  # noqa: F811
    """The records that the binding writes as bytes are those of the structures, field by field."""
    for layout, record in ((H._APPEND_ARGS, H.hsa_append_args), (H._VERIFY_ARGS, H.hsa_verify_args)):
        values = [100 + i for i in range(len(record._fields_))]
        raw = layout.pack(*values)
        assert len(raw) == ctypes.sizeof(record)
        r = record.from_buffer_copy(raw)
        assert [getattr(r, name) for name, _ in record._fields_] == values


def test_rows_on_top_of_one_another(H, monkeypatch):  # noqa: F811
    """Expanded probabilities (rows 0 entries apart) are refused; those of a drafter are not taken for none."""
    monkeypatch.setattr(H, "_stream_on", lambda *_: None)
    i, f = dict(dtype=torch.int32), dict(dtype=torch.float32)
    for nq in (2, 4):
        args = [torch.zeros(2, nq - 1, **i), torch.zeros(2, nq - 1, **f), torch.zeros(2, **f), torch.zeros(2, **i), torch.zeros(2, nq, **i)]
        p, q = torch.zeros(2, nq, 10), torch.zeros(2, nq - 1, 10)
        for a, b in ((p, q[:1, :1].expand(2, nq - 1, 10)), (p[:1, :1].expand(2, nq, 10), q), (p[:1, :1].expand(2, nq, 10), None)):
            with pytest.raises(H.HsaError, match="HSA_ERR_SHAPE"):
                H.hsa_draft_verify(a, b, *args)
