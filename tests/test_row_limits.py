"""The longest rows of scores, on the CPU: the kernels step through a row in 32-bit indices, so
lengths whose last step would pass 2^31 are refused before any launch."""
import ctypes

import pytest

from sparse_attention_indexer_sum_b200 import binding, build

FAKE = ctypes.c_void_p(256)  # never dereferenced: the checks fail first
MOST = 2 ** 31 - 4097


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


@pytest.mark.parametrize("n", [MOST + 1, 2 ** 31 - 1])
def test_topk(lib, n):
    assert lib.ic_topk(FAKE, 1, n, n, -1, 64, FAKE, None) == binding.IC_ERR_UNSUPPORTED
    assert "topk" in binding.ic_last_error()
    assert lib.ic_topk_varlen(FAKE, 1, n, n, FAKE, 64, FAKE, None) == binding.IC_ERR_UNSUPPORTED


@pytest.mark.parametrize("n", [MOST + 1, 2 ** 31 - 1024])
def test_paged_indexer_and_step(lib, n):
    pg = binding.ic_paging(256, 1 << 21, (1 << 21) - 1, 256, 1024, 1)
    st = lib.ic_indexer_scores_paged(FAKE, FAKE, FAKE, FAKE, FAKE, binding.IC_E4M3, 1, 64, 128,
                                     ctypes.byref(pg), n, FAKE, n, None)
    assert st == binding.IC_ERR_UNSUPPORTED and "max_len" in binding.ic_last_error()
    io = binding.ic_layer_io(q_idx=256, q_scale=256, k_idx=256, k_scale=256, w=256, q=256, kv=256,
                             out=256)
    d = binding.make_desc(L=n, k=64, H=64, D=128, idx_dtype=binding.IC_E4M3, heads=16, dk=576,
                          dv=512, attn_dtype=binding.IC_MXF4, scale=1.0, ld_kv=400, batch=1,
                          decode=True)
    st = lib.ic_decode_step_paged(b"F", ctypes.byref(d), ctypes.byref(pg),
                                  (binding.ic_layer_io * 1)(io), 1, FAKE, FAKE, 1 << 40, None)
    assert st == binding.IC_ERR_UNSUPPORTED and "max_len" in binding.ic_last_error()


def test_no_rows_of_the_longest_length_are_fine(lib):
    assert lib.ic_topk(FAKE, 0, MOST, MOST, -1, 64, FAKE, None) == binding.IC_OK


@pytest.mark.parametrize("decode", [False, True])
def test_contiguous_stacks_launch_nothing_for_rows_that_the_topk_refuses(lib, decode):
    io = binding.ic_layer_io(q_idx=256, k_idx=256, w=256, q=256, kv=256, v=256, out=256)
    d = binding.make_desc(L=MOST + 1, k=64, H=1, D=1, idx_dtype=binding.IC_F32, heads=1, dk=1,
                          dv=1, attn_dtype=binding.IC_F32, scale=1.0, batch=1, decode=decode)
    f = lib.ic_decode_step if decode else lib.ic_layer_stack
    st = f(b"F", ctypes.byref(d), (binding.ic_layer_io * 1)(io), 1, FAKE, FAKE, 1 << 40, None)
    assert st == binding.IC_ERR_UNSUPPORTED and "L above the max_len" in binding.ic_last_error()
