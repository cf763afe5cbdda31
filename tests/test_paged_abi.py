"""The paged calls and the norm on the CPU: their argument checks answer before any launch,
and the plain forms that the GPU tests compare with are pinned by hand-worked values."""
import ctypes

import numpy as np
import pytest
import torch

from sparse_attention_indexer_sum_b200 import binding, build
from tests import pagedlib

FAKE = ctypes.c_void_p(256)  # never dereferenced: the checks fail first
ODD = ctypes.c_void_p(257)
INVALID, UNSUPPORTED = binding.IC_ERR_INVALID_ARG, binding.IC_ERR_UNSUPPORTED
BF16, E4M3, F32, MXF4 = binding.IC_BF16, binding.IC_E4M3, binding.IC_F32, binding.IC_MXF4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def _norm(lib, **kw):
    a = dict(x=FAKE, ld_x=64, r=None, ld_r=0, dt=BF16, w=FAKE, w_dt=BF16, eps=1e-6, rows=4, n=64,
             h=None, ld_h=0, y=ctypes.c_void_p(512), ld_y=64, codes=None, ld_c=0, scales=None)
    a.update(kw)
    return lib.ic_rms_norm(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(codes=FAKE, ld_c=64), INVALID), (dict(scales=FAKE), INVALID),
    (dict(dt=E4M3), UNSUPPORTED), (dict(w_dt=MXF4), UNSUPPORTED),
    (dict(n=0), INVALID), (dict(rows=-1), INVALID), (dict(ld_x=63), INVALID),
    (dict(ld_y=63), INVALID), (dict(r=FAKE, ld_r=10), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(x=ODD), INVALID),
    (dict(h=FAKE, ld_h=72), INVALID),                  # h is x with another stride
    (dict(h=ctypes.c_void_p(512), ld_h=64), INVALID),  # h is y
    (dict(rows=1 << 31), UNSUPPORTED),
    (dict(n=(1 << 30) + 1, ld_x=1 << 31, ld_y=1 << 31), UNSUPPORTED),
])
def test_rms_norm_refusals(lib, kw, want):
    assert _norm(lib, **kw) == want
    assert "rms_norm" in binding.ic_last_error()


def test_rms_norm_of_no_rows_launches_nothing(lib):
    assert _norm(lib, rows=0) == binding.IC_OK


def _append(lib, **kw):
    a = dict(rows=4, slots=FAKE, pos=FAKE, rope=FAKE, rope_rows=100, kv=FAKE, ld_kv=576,
             kv_cache=FAKE, ld_cache=576, kv_dt=BF16, k=FAKE, ld_k=128, k_cache=FAKE, k_scale=FAKE,
             k_dt=E4M3, num_slots=64, flags=0)
    a.update(kw)
    return lib.ic_cache_append(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(slots=None), INVALID), (dict(kv=None, k=None), INVALID), (dict(kv_cache=None), INVALID),
    (dict(k_cache=None), INVALID), (dict(pos=None), INVALID), (dict(rows=-1), INVALID),
    (dict(num_slots=0), INVALID), (dict(rope_rows=0), INVALID), (dict(flags=4), INVALID),
    (dict(kv_dt=F32), UNSUPPORTED), (dict(k_dt=MXF4), UNSUPPORTED), (dict(k_scale=None), INVALID),
    (dict(ld_kv=575), INVALID), (dict(ld_kv=580), INVALID), (dict(ld_cache=568), INVALID),
    (dict(kv_dt=E4M3, ld_cache=640), INVALID), (dict(kv_dt=MXF4, ld_cache=399), INVALID),
    (dict(kv_dt=MXF4, ld_cache=408), INVALID), (dict(kv=ctypes.c_void_p(264)), INVALID),
    (dict(k=ctypes.c_void_p(260)), INVALID), (dict(ld_k=126), INVALID), (dict(ld_k=130), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED),
])
def test_cache_append_refusals(lib, kw, want):
    assert _append(lib, **kw) == want
    assert "cache_append" in binding.ic_last_error()


def test_cache_append_of_no_rows_launches_nothing(lib):
    assert _append(lib, rows=0) == binding.IC_OK


def _paging(**kw):
    a = dict(block_table=256, ld_table=8, max_pages=8, seq_lens=256, page_size=64, num_pages=100)
    a.update(kw)
    return binding.ic_paging(**a)


BAD_PAGING = [dict(block_table=None), dict(seq_lens=None), dict(page_size=8), dict(page_size=48),
              dict(page_size=2048), dict(page_size=0), dict(num_pages=0), dict(max_pages=0),
              dict(ld_table=7)]


def _index(lib, pg, **kw):
    a = dict(q=FAKE, qs=FAKE, k=FAKE, ks=FAKE, w=FAKE, dt=E4M3, batch=2, H=64, D=128,
             pg=None if pg is None else ctypes.byref(pg), max_len=512, scores=FAKE, ld=512)
    a.update(kw)
    return lib.ic_indexer_scores_paged(*a.values(), None)


def _attn(lib, pg, **kw):
    a = dict(q=FAKE, kv=FAKE, ld=400, pg=None if pg is None else ctypes.byref(pg), idx=FAKE,
             dt=MXF4, batch=2, rows=1, heads=16, dk=576, dv=512, k=64, scale=1.0, out=FAKE,
             lse=None, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.ic_sparse_attn_paged(*a.values(), None)


@pytest.mark.parametrize("bad", BAD_PAGING)
def test_paging_refusals(lib, bad):
    assert _index(lib, _paging(**bad)) == INVALID
    assert _attn(lib, _paging(**bad)) == INVALID
    d = binding.make_desc(L=512, k=64, H=64, D=128, idx_dtype=E4M3, heads=16, dk=576, dv=512,
                          attn_dtype=MXF4, scale=1.0, ld_kv=400, batch=2, decode=True)
    pg = _paging(**bad)
    arr = (binding.ic_layer_io * 1)()
    assert lib.ic_decode_step_paged(b"F", ctypes.byref(d), ctypes.byref(pg), arr, 1, FAKE, FAKE,
                                    1 << 20, None) == INVALID


def test_paging_of_more_rows_than_32_bits_is_refused(lib):
    assert _index(lib, _paging(num_pages=1 << 26)) == UNSUPPORTED
    assert _attn(lib, _paging(max_pages=1 << 26, ld_table=1 << 26)) == UNSUPPORTED
    assert _attn(lib, None) == INVALID and _index(lib, None) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(w=None), INVALID),
    (dict(scores=None), INVALID), (dict(dt=F32), UNSUPPORTED), (dict(dt=MXF4), UNSUPPORTED),
    (dict(H=32), UNSUPPORTED), (dict(D=64), UNSUPPORTED), (dict(qs=None), INVALID),
    (dict(ks=None), INVALID), (dict(batch=0), INVALID), (dict(max_len=0), INVALID),
    (dict(max_len=513), INVALID), (dict(ld=511), INVALID), (dict(q=ctypes.c_void_p(264)), INVALID),
])
def test_indexer_paged_refusals(lib, kw, want):
    assert _index(lib, _paging(), **kw) == want
    assert "indexer_paged" in binding.ic_last_error()


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(kv=None), INVALID), (dict(idx=None), INVALID),
    (dict(out=None), INVALID), (dict(dt=F32), UNSUPPORTED), (dict(heads=8), UNSUPPORTED),
    (dict(dk=512), UNSUPPORTED), (dict(dv=576), UNSUPPORTED), (dict(k=0), INVALID),
    (dict(k=2049), UNSUPPORTED), (dict(batch=0), INVALID), (dict(rows=-1), INVALID),
    (dict(ld=399), INVALID), (dict(ld=408), INVALID), (dict(dt=E4M3), INVALID),
    (dict(dt=BF16), INVALID), (dict(kv=ctypes.c_void_p(264)), INVALID),
])
def test_attn_paged_refusals(lib, kw, want):
    assert _attn(lib, _paging(), **kw) == want
    assert "attn_paged" in binding.ic_last_error()


def test_4bit_rows_are_refused_where_only_pages_have_them(lib):
    st = lib.ic_sparse_attn(FAKE, FAKE, 400, None, FAKE, MXF4, 1, 4, 16, 576, 512, 100, 64, 1.0,
                            FAKE, None, None, 0, None)
    assert st in (INVALID, UNSUPPORTED)


def test_decode_step_paged_refusals(lib):
    pg = _paging()
    io = binding.ic_layer_io(q_idx=256, q_scale=256, k_idx=256, k_scale=256, w=256, q=256, kv=256,
                             out=256)

    def call(pattern=b"F", layers=1, ws=1 << 20, io=io, **kw):
        a = dict(L=512, k=64, H=64, D=128, idx_dtype=E4M3, heads=16, dk=576, dv=512,
                 attn_dtype=MXF4, scale=1.0, ld_kv=400, batch=2, decode=True)
        a.update(kw)
        d = binding.make_desc(**a)
        arr = (binding.ic_layer_io * 1)(io)
        return lib.ic_decode_step_paged(pattern, ctypes.byref(d), ctypes.byref(pg), arr, layers,
                                        FAKE, FAKE, ws, None)

    assert call(pattern=b"S") == INVALID
    assert call(pattern=b"F,S") == INVALID
    assert call(decode=False) == INVALID
    assert call(flags=binding.IC_STACK_FUSED_TOPK) == UNSUPPORTED
    assert call(L=513) == INVALID                       # past max_pages * page_size
    assert call(idx_dtype=F32) == UNSUPPORTED
    assert call(attn_dtype=F32) == UNSUPPORTED
    assert call(k=4096) == INVALID
    assert call(ws=512 * 4 - 1) == binding.IC_ERR_WORKSPACE
    assert call(io=binding.ic_layer_io(q_idx=256, q_scale=256, k_idx=256, k_scale=256, w=256,
                                       q=256, kv=256, v=256, out=256)) == UNSUPPORTED
    assert "layer 0" in binding.ic_last_error()


def test_binding_refuses_before_the_library_is_called():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        binding.ic_rms_norm(x, w)
    with pytest.raises(ValueError, match="weight"):
        binding.ic_rms_norm(x, w[:32])
    with pytest.raises(ValueError, match="evenly"):
        binding.ic_rms_norm(torch.zeros(4, 3, 128, dtype=torch.bfloat16)[:, :2, :64], w)
    s = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        binding.ic_cache_append(s.int(), k=x, k_cache=x)
    t, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="block_table"):
        binding.make_paging(t.long(), n, 64, 10)
    with pytest.raises(ValueError, match="seq_lens"):
        binding.make_paging(t, n[:1], 64, 10)
    with pytest.raises(ValueError, match="contiguous rows"):
        binding.make_paging(t.t(), torch.zeros(4, dtype=torch.int32), 64, 10)


def test_rope_table_keeps_far_angles():
    t = binding.rope_table(200001)
    for p, i in ((0, 0), (1, 0), (199999, 0), (200000, 31), (123456, 7)):
        a = p * 10000.0 ** (-i / 32)
        assert abs(t[p, i].item() - np.cos(a)) < 2 ** -23
        assert abs(t[p, 32 + i].item() - np.sin(a)) < 2 ** -23


def test_plain_mxf4_rows_by_hand():
    x = np.zeros((1, 576))
    # block 0: largest 6 -> scale 1; every tie goes to the even code
    x[0, :10] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.2, -6.0]
    x[0, 32] = 6.5         # block 1: above 6 -> scale 2: 3.25 -> 3
    x[0, 64] = 2.0 ** -10  # block 2: m = 1 -> 2^-12, code 6 (4.0)
    x[0, 575] = 1.5
    row = pagedlib.pack_mxf4(x)[0]
    codes = [row[i // 2] >> (4 * (i % 2)) & 15 for i in range(10)]
    assert codes == [7, 0, 2, 2, 4, 4, 6, 6, 8, 15]
    assert row[256] == 127 and row[257] == 128 and row[16] & 15 == 5
    assert row[258] == 127 - 12 and row[32] & 15 == 6
    assert row[259] == 0 and row[398] == 0xC0 and row[399] == 0x3F
    back = pagedlib.unpack(torch.from_numpy(row), "mxf4")
    assert back[0] == 6.0 and back[9] == -6.0 and back[32] == 6.0 and back[64] == 2.0 ** -10
    assert back[575] == 1.5
