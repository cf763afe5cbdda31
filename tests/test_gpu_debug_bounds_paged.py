"""The debug-bounds build on the paged calls: what their documentation allows (entries past a
sequence's length, tokens without a slot or with a position outside the table, lengths of 0)
is no finding, a page number outside the pool is one; results are the release build's."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from sparse_attention_indexer_sum_b200 import binding as ic
from sparse_attention_indexer_sum_b200 import build
from tests import pagedlib

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KINDS = {"bf16": ic.IC_BF16, "e4m3": ic.IC_E4M3, "mxf4": ic.IC_MXF4}
WIDTH = {"bf16": 576, "e4m3": 656, "mxf4": 400}
LENS, PAGE = [300, 0, 70], 32

CHILD = r"""
import json, sys
import numpy as np
sys.path.insert(0, sys.argv[1])
from tests.test_gpu_debug_bounds_paged import cases, status
out = {}
for name, f in cases():
    for i, t in enumerate(f()):
        np.save("%s_%s_%d.npy" % (sys.argv[2], name, i), t)
    out[name] = status()
print(json.dumps(out))
"""


def status():
    try:
        ic.ic_device_status()
    except ic.ICError as e:
        return e.status
    return 0


def _append(kind):
    g = torch.Generator().manual_seed(1)
    n, pages = 400, 14
    kv = torch.randn(n, 576, generator=g).bfloat16()
    k = torch.randn(n, 128, generator=g).bfloat16()
    slots = torch.randperm(pages * PAGE, generator=g)[:n]
    slots[3], slots[40], slots[77] = -1, pages * PAGE, 1 << 40
    pos = torch.randint(0, 500, (n,), generator=g, dtype=torch.int32)
    pos[5], pos[6] = -3, 500
    c = torch.zeros(pages, PAGE, WIDTH[kind], dtype=torch.bfloat16 if kind == "bf16" else torch.uint8,
                    device=DEV)
    kc = torch.zeros(pages, PAGE, 128, dtype=torch.uint8, device=DEV)
    ks = torch.zeros(pages, PAGE, device=DEV)
    ic.ic_cache_append(slots.to(DEV), kv=kv.to(DEV), kv_cache=c, kv_dtype=KINDS[kind], k=k.to(DEV),
                       k_cache=kc, k_scale=ks, pos=pos.to(DEV), rope=ic.rope_table(500, device=DEV))
    return c, kc, ks


def _paged(kind, bad):
    g = torch.Generator().manual_seed(2)
    c, kc, ks = _append(kind)
    table, pages = pagedlib.shuffled_table(LENS, PAGE, 1, g)
    if bad:
        table[0, 2] = 1 << 20
    q = torch.randn(3, 2, 16, 576, generator=g).bfloat16().to(DEV)
    idx = torch.randint(-1, 320, (3, 2, 64), generator=g, dtype=torch.int32)  # past every length
    idx[0, 0, 5] = -9
    idx[0, 1, 0] = 64                    # the page that `bad` breaks
    sl = torch.tensor(LENS, dtype=torch.int32, device=DEV)
    out = ic.ic_sparse_attn_paged(q, c, idx.to(DEV), table.to(DEV), sl, 0.04, page_size=PAGE,
                                  kv_dtype=KINDS[kind])
    return out


def _scores(bad):
    g = torch.Generator().manual_seed(3)
    _, kc, ks = _append("bf16")
    table, _ = pagedlib.shuffled_table(LENS, PAGE, 1, g)
    if bad:
        table[2, 1] = -7
    q8, qs = ic.ic_quant_e4m3_rows(torch.randn(3, 64, 128, generator=g).bfloat16().to(DEV))
    w = torch.rand(3, 64, generator=g).to(DEV)
    s = torch.zeros(3, 320, device=DEV)
    ic.ic_indexer_scores_paged(q8, kc, w, table.to(DEV), torch.tensor(LENS, dtype=torch.int32,
                                                                     device=DEV),
                               page_size=PAGE, scores=s, q_scale=qs, k_scale=ks)
    return s


def _np(*ts):
    torch.cuda.synchronize()
    return [t.float().cpu().numpy() for t in ts]


def cases():
    for kind in KINDS:
        yield "append_" + kind, lambda kind=kind: _np(*_append(kind))
        for bad in (False, True):
            yield "attn_%s%s" % (kind, "_bad" * bad), lambda kind=kind, bad=bad: _np(_paged(kind, bad))
    for bad in (False, True):
        yield "scores" + "_bad" * bad, lambda bad=bad: _np(_scores(bad))


def test_legal_inputs_report_nothing_and_a_page_outside_the_pool_does(tmp_path):
    build.build(debug_bounds=True)
    env = dict(os.environ, IC_DEBUG_BOUNDS="1", PYTHONPATH=ROOT)
    base = str(tmp_path / "dbg")
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, base], env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    st = json.loads(r.stdout.strip().splitlines()[-1])
    assert st == {name: ic.IC_ERR_BOUNDS if name.endswith("_bad") else 0 for name, _ in cases()}
    for name, f in cases():
        for i, t in enumerate(f()):
            assert np.array_equal(np.load("%s_%s_%d.npy" % (base, name, i)), t, equal_nan=True), name
        assert status() == 0
