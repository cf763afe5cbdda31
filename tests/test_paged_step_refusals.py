"""What the paged decode step's binding refuses before anything is launched (no GPU): host
tensors, and tensors that hold less than the description and the paging name."""
import pytest
import torch

from sparse_attention_indexer_sum_b200 import binding as ic

B, PAGE, PAGES, K = 3, 16, 5, 32


def _case(kv_dtype=ic.IC_MXF4, idx_dtype=ic.IC_E4M3, **over):
    """(desc, paging, layers, t_cache, workspace) of a step that fits; `over` replaces tensors
    of layer 0."""
    width = {ic.IC_BF16: 576, ic.IC_E4M3: 656, ic.IC_MXF4: 400}[kv_dtype]
    fp8 = idx_dtype == ic.IC_E4M3
    it = torch.uint8 if fp8 else torch.bfloat16
    layers = []
    for _ in range(2):
        layers.append(dict(
            q_idx=torch.zeros(B, 1, 64, 128, dtype=it), w=torch.zeros(B, 1, 64),
            q_scale=torch.zeros(B, 1, 64) if fp8 else None,
            k_idx=torch.zeros(PAGES, PAGE, 128, dtype=it),
            k_scale=torch.zeros(PAGES, PAGE) if fp8 else None,
            q=torch.zeros(B, 1, 16, 576, dtype=torch.bfloat16),
            kv=torch.zeros(PAGES, PAGE, width,
                           dtype=torch.bfloat16 if kv_dtype == ic.IC_BF16 else torch.uint8),
            out=torch.zeros(B, 1, 16, 512, dtype=torch.bfloat16), lse=torch.zeros(B, 1, 16)))
    layers[0].update(over)
    table = torch.zeros(B, 4, dtype=torch.int32)
    lens = torch.ones(B, dtype=torch.int32)
    paging = ic.ic_paging(table.data_ptr(), 4, 4, lens.data_ptr(), PAGE, PAGES)
    paging.tensors = (table, lens)
    desc = ic.make_desc(L=64, k=K, H=64, D=128, idx_dtype=idx_dtype, heads=16, dk=576, dv=512,
                        attn_dtype=kv_dtype, scale=1.0, ld_kv=width, batch=B, decode=True)
    return desc, paging, layers, torch.zeros(B, K, dtype=torch.int32), torch.zeros(B * 64)


def _step(desc, paging, layers, t_cache, ws, pattern="F,S"):
    ic.ic_decode_step_paged(pattern, desc, paging, layers, t_cache, ws)


@pytest.mark.parametrize("kv_dtype", [ic.IC_BF16, ic.IC_E4M3, ic.IC_MXF4])
@pytest.mark.parametrize("idx_dtype", [ic.IC_BF16, ic.IC_E4M3])
def test_host_tensors(kv_dtype, idx_dtype):
    with pytest.raises(ValueError, match="CUDA device"):
        _step(*_case(kv_dtype, idx_dtype))
    with pytest.raises(ValueError, match="CUDA device"):
        ic.make_paging(torch.zeros(B, 4, dtype=torch.int32), torch.ones(B, dtype=torch.int32),
                       PAGE, PAGES)


def test_a_batch_larger_than_the_block_table_or_the_index_cache():
    desc, paging, layers, t, ws = _case()
    desc.batch = B + 1
    with pytest.raises(ValueError, match="block table has 3 rows"):
        _step(desc, paging, layers, t, ws)
    paging.tensors = ()          # a table that the binding does not know: the others are checked
    with pytest.raises(ValueError, match="t_cache"):
        _step(desc, paging, layers, t, ws)


def test_a_smaller_batch_than_the_tensors_hold_fits():
    desc, paging, layers, t, ws = _case()
    desc.batch = B - 1
    with pytest.raises(ValueError, match="CUDA device"):  # nothing else is wrong
        _step(desc, paging, layers, t, ws)


@pytest.mark.parametrize("name,t", [
    ("t_cache", torch.zeros(B, K, dtype=torch.int64)), ("t_cache", torch.zeros(B, K - 1).int()),
    ("t_cache", torch.zeros(B, 2 * K, dtype=torch.int32)[:, ::2])])
def test_index_cache(name, t):
    desc, paging, layers, _, ws = _case()
    with pytest.raises(ValueError, match=name):
        _step(desc, paging, layers, t, ws)


BF = torch.bfloat16
BAD = [
    ("k_idx", torch.zeros(PAGES - 1, PAGE, 128, dtype=torch.uint8)),
    ("k_idx", torch.zeros(PAGES, PAGE, 128, dtype=BF)),
    ("k_idx", torch.zeros(PAGES, PAGE, 256, dtype=torch.uint8)[..., :128]),
    ("k_scale", torch.zeros(PAGES * PAGE - 1)), ("k_scale", torch.zeros(PAGES, PAGE).double()),
    ("q_idx", torch.zeros(B - 1, 64, 128, dtype=torch.uint8)),
    ("q_scale", torch.zeros(B, 63)), ("w", torch.zeros(B, 64, dtype=BF)),
    ("q", torch.zeros(B, 16, 575, dtype=BF)), ("q", torch.zeros(B, 16, 576)),
    ("out", torch.zeros(B, 16, 511, dtype=BF)), ("lse", torch.zeros(B, 15)),
    ("kv", torch.zeros(PAGES - 1, PAGE, 400, dtype=torch.uint8)),
    ("kv", torch.zeros(PAGES, PAGE, 400, dtype=BF)),
    ("kv", torch.zeros(PAGES, PAGE, 416, dtype=torch.uint8)[..., :400]),      # another stride
    ("kv", torch.zeros(PAGES, 2 * PAGE, 400, dtype=torch.uint8)[:, :PAGE]),   # gaps
]


@pytest.mark.parametrize("name,t", BAD, ids=["%s-%d" % (n, i) for i, (n, _) in enumerate(BAD)])
def test_layer_tensors(name, t):
    with pytest.raises(ValueError, match=r"layer 0: %s\b" % name):
        _step(*_case(**{name: t}))


def test_tensors_that_a_shared_layer_does_not_use_are_not_looked_at():
    desc, paging, layers, t, ws = _case()
    layers[1].update(k_idx=torch.zeros(1), q_idx=None, w=torch.zeros(2), k_scale=None)
    with pytest.raises(ValueError, match="CUDA device"):
        _step(desc, paging, layers, t, ws)


def test_longer_rows_and_flat_pools_fit():
    desc, paging, layers, t, ws = _case(
        kv=torch.zeros(PAGES, PAGE, 432, dtype=torch.uint8)[..., :416])
    layers[1]["kv"] = torch.zeros(PAGES * PAGE * 432, dtype=torch.uint8)
    desc.ld_kv = 432
    with pytest.raises(ValueError, match="CUDA device"):
        _step(desc, paging, layers, t, ws)


def test_a_workspace_with_gaps():
    desc, paging, layers, t, _ = _case()
    with pytest.raises(ValueError, match="contiguous"):
        _step(desc, paging, layers, t, torch.zeros(B * 64, 2)[:, 0])


def test_make_paging_keeps_its_tensors():
    """(the object is what a captured step reads through)"""
    table, lens = torch.zeros(B, 4, dtype=torch.int32), torch.ones(B, dtype=torch.int32)
    real = ic._one_device
    try:
        ic._one_device = lambda *ts: 0
        pg = ic.make_paging(table, lens, PAGE, PAGES)
    finally:
        ic._one_device = real
    assert pg.tensors[0] is table and pg.tensors[1] is lens
    assert pg.block_table == table.data_ptr() and pg.max_pages == 4
