"""Attention over selected rows that are not finite, in every form of the call, against the
formula in 64 bits: the log of the sum is NaN with a NaN score, +inf with a score of +inf,
and -inf for a query without entries alone."""
import math

import pytest
import torch

from sparse_attention_indexer_sum_b200 import binding as ic

pytestmark = pytest.mark.gpu
DEV = "cuda"
KINDS = {"bf16": ic.IC_BF16, "e4m3": ic.IC_E4M3, "mxf4": ic.IC_MXF4}
WIDTH = {"bf16": 576, "e4m3": 656, "mxf4": 400}
U_BF16, U_F32 = 2.0 ** -8, 2.0 ** -24


def _rows(n, g):
    """Latent rows: 0 has a NaN, 1 a +inf in a rope dim that only heads 0..7 look at, the
    others are finite (and exact in every format: small integers)."""
    x = torch.randint(-3, 4, (n, 576), generator=g).float()
    x[0, 3] = math.nan
    x[1, 575] = math.inf
    return x.bfloat16()


def _queries(R, g):
    q = torch.randint(-2, 3, (1, R, 16, 576), generator=g).float()
    q[..., 575] = 0.0
    q[:, :, :8, 575] = 1.0
    return q.bfloat16()


def _lists(R, n, k, g):
    """Query r's entries by r % 5: finite rows, row 0 alone, rows with 0, rows with 1, none."""
    idx = torch.full((1, R, k), -1, dtype=torch.int32)
    for r in range(R):
        m = (k, 1, k - 3, k // 2, 0)[r % 5]
        idx[0, r, :m] = (2 + torch.randperm(n - 2, generator=g)[:m]).int()
        if r % 5 == 1:
            idx[0, r, 0] = 0
        if r % 5 == 2:
            idx[0, r, m // 2] = 0
        if r % 5 == 3:
            idx[0, r, m - 1] = 1
    return idx


def _check(q, x, idx, scale, out, lse, v=None):
    """q, x, idx as given to the call (x: the values that the cache's rows stand for)."""
    H = q.shape[2]
    V = x[:, :512] if v is None else v
    for r in range(idx.shape[1]):
        t = idx[0, r].long()
        t = t[t >= 0]
        o, l = out[0, r].double().cpu(), lse[0, r].double().cpu()
        if t.numel() == 0:
            assert (o == 0).all() and torch.isneginf(l).all(), r
            continue
        z = q[0, r].double() @ x[t].double().T * scale
        if r % 5 == 3:            # 0 * inf of the heads that do not look at the infinity
            assert torch.isnan(z[8:]).any(1).all() and torch.isposinf(z[:8]).any(1).all()
        want = torch.logsumexp(z, -1)
        ref = torch.softmax(z, -1) @ V[t].double()
        for h in range(H):
            if torch.isfinite(want[h]):
                # logits are exact here (small integers); their scaling, the exponentials and
                # the sums round in fp32, probabilities and outputs to bf16
                assert abs(l[h] - want[h]) <= 1e-5 + 8 * U_F32 * want[h].abs(), (r, h)
                spread = torch.softmax(z[h], -1) @ V[t].double().abs()
                lim = (U_BF16 + 1e-4) * spread + U_BF16 * ref[h].abs()
                assert ((o[h] - ref[h]).abs() <= lim * (1 + U_BF16)).all(), (r, h)
            else:
                assert torch.equal(torch.isnan(l[h]), torch.isnan(want[h])), (r, h, l[h], want[h])
                assert torch.isnan(want[h]) or l[h] == want[h], (r, h)
                assert torch.isnan(o[h]).all(), (r, h)


# few queries are split over several CTAs where there is a workspace; 700 are not
@pytest.mark.parametrize("R,k", [(5, 200), (10, 64), (700, 70)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxf4"])
@pytest.mark.parametrize("ws", [False, True])
def test_paged(kind, R, k, ws):
    g = torch.Generator().manual_seed(R)
    n, page = 256, 32
    x, q, idx = _rows(n, g), _queries(R, g), _lists(R, n, k, g)
    cache = x.to(DEV)
    if kind != "bf16":
        cache = torch.zeros(n, WIDTH[kind], dtype=torch.uint8, device=DEV)
        ic.ic_cache_append(torch.arange(n, device=DEV), kv=x.to(DEV), kv_cache=cache,
                           kv_dtype=KINDS[kind])
    from tests import pagedlib
    values = pagedlib.unpack(cache, kind).cpu()
    table = torch.arange(n // page, dtype=torch.int32, device=DEV)[None]
    lse = torch.zeros(1, R, 16, device=DEV)
    work = torch.empty(ic.ic_attn_workspace_size(1, R, 16, 512, k) + 16, dtype=torch.uint8,
                       device=DEV)
    out = ic.ic_sparse_attn_paged(q.to(DEV), cache, idx.to(DEV), table,
                                  torch.tensor([n], dtype=torch.int32, device=DEV), 0.01,
                                  page_size=page, kv_dtype=KINDS[kind], lse=lse,
                                  workspace=work if ws else None)
    ic.ic_device_status()
    _check(q, values, idx, 0.01, out, lse)


@pytest.mark.parametrize("R,k", [(5, 200), (10, 64)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("ws", [False, True])
def test_contiguous(kind, R, k, ws):
    g = torch.Generator().manual_seed(R + 1)
    n = 256
    x, q, idx = _rows(n, g), _queries(R, g), _lists(R, n, k, g)
    cache = x.to(DEV) if kind == "bf16" else ic.ic_pack_kv_e4m3(x.to(DEV))
    from tests import pagedlib
    values = pagedlib.unpack(cache, kind).cpu()
    lse = torch.zeros(1, R, 16, device=DEV)
    work = torch.empty(ic.ic_attn_workspace_size(1, R, 16, 512, k) + 16, dtype=torch.uint8,
                       device=DEV)
    out = ic.ic_sparse_attn(q.to(DEV), cache[None], idx.to(DEV), 0.01, lse=lse,
                            workspace=work if ws else None)
    ic.ic_device_status()
    _check(q, values, idx, 0.01, out, lse)


def test_fp32_with_separate_values():
    g = torch.Generator().manual_seed(7)
    n, R, k = 60, 10, 20
    x = torch.randint(-3, 4, (n, 64), generator=g).float()
    x[0, 3] = math.nan
    x[1, 63] = math.inf
    q = torch.randint(-2, 3, (1, R, 4, 64), generator=g).float()
    q[..., 63] = 1.0                     # every head meets the infinity
    v = torch.randn(n, 48, generator=g)
    idx = _lists(R, n, k, g)
    lse = torch.zeros(1, R, 4, device=DEV)
    out = ic.ic_sparse_attn(q.to(DEV), x[None].to(DEV), idx.to(DEV), 0.1, v=v[None].to(DEV),
                            lse=lse)
    ic.ic_device_status()
    for r in range(R):
        t = idx[0, r].long()
        t = t[t >= 0]
        z = q[0, r].double() @ x[t].double().T * 0.1
        want = torch.logsumexp(z, -1) if t.numel() else torch.full((4,), -math.inf).double()
        l, o = lse[0, r].double().cpu(), out[0, r].double().cpu()
        if torch.isfinite(want).all():
            ref = torch.softmax(z, -1) @ v[t].double()
            assert ((l - want).abs() <= 1e-5 + 16 * U_F32 * want.abs()).all()
            # 64 products, the exponential and 20 terms of a sum, one fp32 step each
            lim = (120 * U_F32 + 1e-6) * (torch.softmax(z, -1) @ v[t].double().abs())
            assert ((o - ref).abs() <= lim).all()
        elif t.numel() == 0:
            assert torch.isneginf(l).all() and (o == 0).all()
        else:
            assert torch.equal(torch.isnan(l), torch.isnan(want)) and torch.isnan(o).all()
            assert (torch.isnan(want) | (l == want)).all()


# -------------------------------------------- rows of one query do not reach another
def _mixed_lists(R, n, k, g):
    """Every third query selects rows 0..63 (which the tests fill with NaN and infinities),
    the others fewer rows of the rest, so that their tiles keep places without a row."""
    idx = torch.full((1, R, k), -1, dtype=torch.int32)
    idx[0, 0::3, :64] = torch.arange(64, dtype=torch.int32)
    for r in range(R):
        if r % 3:
            m = r % 40
            idx[0, r, :m] = (64 + torch.randperm(n - 64, generator=g)[:m]).int()
    return idx


@pytest.mark.parametrize("R,ws", [(700, False), (300, True)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_contiguous_rows_stay_with_their_query(kind, R, ws):
    g = torch.Generator().manual_seed(R)
    n, k = 256, 64
    x = torch.randn(n, 576, generator=g).bfloat16()
    idx = _mixed_lists(R, n, k, g).to(DEV)
    q = torch.randn(1, R, 16, 576, generator=g).bfloat16().to(DEV)
    work = torch.empty(ic.ic_attn_workspace_size(1, R, 16, 512, k) + 16, dtype=torch.uint8,
                       device=DEV) if ws else None
    got = []
    for bad in (False, True):
        if bad:
            x[0:64:2] = math.inf
            x[1:64:2] = math.nan
        cache = x.to(DEV) if kind == "bf16" else ic.ic_pack_kv_e4m3(x.to(DEV))
        lse = torch.zeros(1, R, 16, device=DEV)
        got.append((ic.ic_sparse_attn(q, cache[None], idx, 0.04, lse=lse, workspace=work), lse))
        ic.ic_device_status()
    others = [r for r in range(R) if r % 3]
    for a, b in zip(*got):
        assert torch.equal(a[0, others], b[0, others])
    assert torch.isfinite(got[0][0]).all() and torch.isnan(got[1][0][0, 0::3]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_packed_sequences_rows_stay_with_their_sequence(fp8):
    """Three sequences in shared launches; the first one's cache rows become NaN and inf."""
    from tests.test_gpu_parity import _varlen_mla_case
    lens = [400, 300, 333]
    wl0, per, packed, desc = _varlen_mla_case(lens, "F,S", False, seed=3)
    desc.attn_dtype = ic.IC_E4M3 if fp8 else ic.IC_BF16
    desc.ld_kv = ic.KV8_ROW_BYTES if fp8 else 576
    cu = [0, 400, 700, 1033]
    ws = torch.empty(1033 * (wl0.L + 1) + 64, device=DEV)
    got = []
    for bad in (False, True):
        t = torch.full((1033, wl0.k), -7, dtype=torch.int32, device=DEV)
        layers = []
        for e in packed:
            kv = e["kv"].clone()
            if bad:
                kv[0:400:2] = math.inf
                kv[1:400:2] = math.nan
            layers.append(dict(e, kv=ic.ic_pack_kv_e4m3(kv) if fp8 else kv,
                               out=torch.empty_like(e["out"]), lse=torch.empty_like(e["lse"])))
        ic.ic_layer_stack_varlen("F,S", desc, layers, cu, t, ws)
        ic.ic_device_status()
        got.append((t, [e["out"] for e in layers], [e["lse"] for e in layers]))
    assert torch.equal(got[0][0], got[1][0])
    for l in range(2):
        for a, b in zip(got[0][1:], got[1][1:]):
            assert torch.equal(a[l][400:], b[l][400:]) and torch.isfinite(a[l][400:]).all()
        assert torch.isnan(got[1][1][l][:400]).all()
