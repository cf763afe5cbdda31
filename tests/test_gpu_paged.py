"""The norm, the cache append and the paged indexer, attention and decode step on the GPU
against plain 64-bit forms.

Tolerances follow from the arithmetic: u(t) = finfo(t).eps / 2 is half a step of type t.
An fp32 sum of positive terms along a chain of m additions is off by at most m u(f32)
relative; the tensor cores' fp32 sums are counted at one whole step per addition.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from sparse_attention_indexer_sum_b200 import binding as ic
from tests import pagedlib

pytestmark = pytest.mark.gpu
DEV = "cuda"
U_BF16, U_F32, U_E4M3 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4
KINDS = {"bf16": ic.IC_BF16, "e4m3": ic.IC_E4M3, "mxf4": ic.IC_MXF4}
WIDTH = {"bf16": 576, "e4m3": 656, "mxf4": 400}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------------------- RMS norm
def _check_norm(x, r, w, eps, h, y, codes, scales):
    """x, r, w as given to the kernel, outputs as it left them (any may be None)."""
    n = x.shape[-1]
    hd = x.double() + (0 if r is None else r.double())
    rstd = 1 / (hd.pow(2).mean(-1, keepdim=True) + eps).sqrt()
    ref = hd * rstd * w.double()
    # the sum: n / 256 + 11 additions at most (halved by the root), the addition x + r, the
    # root (2 steps) and two products; the products' results round once more below
    rel = ((n / 256 + 11) / 2 + 8) * U_F32
    slop = rel * ref.abs() + U_F32 * (x.double().abs() + (0 if r is None else r.double().abs())) * \
        (rstd * w.double()).abs() + 1e-37
    if h is not None:
        u = torch.finfo(h.dtype).eps / 2
        assert ((h.double() - hd).abs() <= (u + 2 * U_F32) * hd.abs() + 1e-38).all()
    if y is not None:
        u = torch.finfo(y.dtype).eps / 2
        err = (y.double() - ref).abs()
        assert (err <= u * ref.abs() + slop * (1 + u)).all(), (err - u * ref.abs() - slop).max()
    if codes is not None:
        m = -(-n // 128)
        pad = torch.nn.functional.pad(ref, (0, m * 128 - n)).unflatten(-1, (m, 128))
        want = pad.abs().amax(-1) / 448
        want[want == 0] = 1.0
        slop_g = torch.nn.functional.pad(slop, (0, m * 128 - n)).unflatten(-1, (m, 128))
        assert ((scales.double() - want).abs() <=
                slop_g.amax(-1) / 448 + 4 * U_F32 * want + 1e-38).all()
        sc = scales.double().repeat_interleave(128, -1)[..., :n]
        val = codes.view(torch.float8_e4m3fn).float().double()
        q = (ref / sc).clamp(-448, 448)
        lim = pagedlib.e4m3_half_step(q) * (1 + 1e-9) + (slop / sc + 4 * U_F32 * q.abs()) * 1.01
        # a value next to a power of two may round on the coarser side of it
        lim = torch.maximum(lim, pagedlib.e4m3_half_step(val))
        assert ((val - q).abs() <= lim + 4 * U_F32 * q.abs() + slop / sc).all()


@pytest.mark.parametrize("n", [1, 7, 8, 100, 128, 136, 512, 1000, 4096, 4104, 5000, 8192, 8200,
                               16384, 16392, 20001])
@pytest.mark.parametrize("dt,wdt,res", [(torch.bfloat16, torch.bfloat16, True),
                                        (torch.float32, torch.float32, True),
                                        (torch.bfloat16, torch.float32, False),
                                        (torch.float32, torch.bfloat16, False)])
def test_rms_norm(n, dt, wdt, res):
    g = _gen(n)
    rows = 5
    x = torch.randn(rows, n, generator=g).to(dt).to(DEV)
    r = (3 * torch.randn(rows, n, generator=g)).to(dt).to(DEV) if res else None
    w = (1 + 0.2 * torch.randn(n, generator=g)).to(wdt).to(DEV)
    h, y = torch.empty_like(x), torch.empty_like(x)
    codes = torch.empty(rows, n, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, -(-n // 128), device=DEV)
    ic.ic_rms_norm(x, w, 1e-5, residual=r, h=h, y=y, codes=codes, scales=scales)
    ic.ic_device_status()
    _check_norm(x, r, w, 1e-5, h, y, codes, scales)
    # each output alone is the same bits
    y2, _, _ = ic.ic_rms_norm(x, w, 1e-5, residual=r)
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    ic.ic_rms_norm(x, w, 1e-5, residual=r, codes=c2, scales=s2)
    assert torch.equal(y, y2) and torch.equal(codes, c2) and torch.equal(scales, s2)


@pytest.mark.parametrize("off,ld", [(0, 576), (8, 584), (1, 577), (3, 600), (4, 580)])
def test_rms_norm_strided_rows_and_neighbours(off, ld):
    """The latent part of [rows, ld] rows normalised where it lies; other columns stay."""
    g = _gen(ld + off)
    full = torch.randn(37, ld, generator=g).bfloat16().to(DEV)
    keep = full.clone()
    x = full[:, off:off + 512]
    w = torch.rand(512, generator=g).to(DEV)
    codes = torch.full((37, 530), 255, dtype=torch.uint8, device=DEV)
    scales = torch.empty(37, 4, device=DEV)
    ic.ic_rms_norm(x, w, 1e-6, y=x, codes=codes[:, 9:521], scales=scales)
    ic.ic_device_status()
    _check_norm(keep[:, off:off + 512], None, w, 1e-6, None, x, codes[:, 9:521].contiguous(),
                scales)
    assert torch.equal(full[:, :off], keep[:, :off])
    assert torch.equal(full[:, off + 512:], keep[:, off + 512:])
    assert (codes[:, :9] == 255).all() and (codes[:, 521:] == 255).all()


@pytest.mark.parametrize("n", [1024, 1023])
def test_rms_norm_in_place_residual(n):
    g = _gen(5)
    x = torch.randn(9, n, generator=g).bfloat16().to(DEV)
    r = torch.randn(9, n, generator=g).bfloat16().to(DEV)
    w = torch.ones(n, device=DEV)
    x0, r0 = x.clone(), r.clone()
    ic.ic_rms_norm(x, w, 1e-6, residual=r, h=r, y=x)
    ic.ic_device_status()
    _check_norm(x0, r0, w, 1e-6, r, x, None, None)


@pytest.mark.parametrize("n", [512, 509])
def test_rms_norm_zero_rows_and_non_finite_rows(n):
    x = torch.randn(6, n, generator=_gen(1)).bfloat16()
    x[1] = 0.0
    x[2, 3] = math.nan
    x[3, 5] = math.inf
    x = x.to(DEV)
    w = torch.ones(n, device=DEV)
    codes = torch.empty(6, n, dtype=torch.uint8, device=DEV)
    scales = torch.empty(6, -(-n // 128), device=DEV)
    y, _, _ = ic.ic_rms_norm(x, w, 1e-6)
    ic.ic_rms_norm(x, w, 1e-6, codes=codes, scales=scales)
    ic.ic_device_status()
    for i in (0, 4, 5):
        _check_norm(x[i:i + 1], None, w, 1e-6, None, y[i:i + 1], codes[i:i + 1], scales[i:i + 1])
    assert (y[1] == 0).all() and (codes[1] == 0).all() and (scales[1] == 1).all()
    assert torch.isnan(y[2]).all() and torch.isnan(y[3, 5])


def test_rms_norm_of_no_rows():
    y, _, _ = ic.ic_rms_norm(torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV))
    assert y.shape == (0, 64)


def test_rms_norm_of_large_values_and_many_rows():
    x = (1e6 * torch.randn(3000, 264, generator=_gen(2))).to(DEV)
    w = torch.randn(264, generator=_gen(3)).to(DEV)
    y, _, _ = ic.ic_rms_norm(x, w, 0.0)
    ic.ic_device_status()
    _check_norm(x, None, w, 0.0, None, y, None, None)


# ------------------------------------------------------------------------------- append
def _caches(kind, kdt, pages, page, pad=0):
    dt = torch.bfloat16 if kind == "bf16" else torch.uint8
    kv = torch.full((pages, page, WIDTH[kind] + pad), 7, dtype=dt, device=DEV)
    k = torch.full((pages, page, 128), 7, dtype=torch.bfloat16 if kdt == "bf16" else torch.uint8,
                   device=DEV)
    return kv, k, torch.full((pages, page), 7.0, device=DEV) if kdt == "e4m3" else None


def _check_latent(got, x, kind, cos, sin, halves):
    """got [n, width] of x [n, 576] bf16 (CPU tensors)."""
    if kind == "mxf4":
        want = pagedlib.pack_mxf4(x.double().numpy())
        np.testing.assert_array_equal(got[:, :272].numpy(), want[:, :272])
        tail = got[:, 272:400].contiguous().view(torch.bfloat16)
    elif kind == "e4m3":
        codes, scales, _ = oracle.kv_pack_e4m3(x.float().numpy())
        np.testing.assert_array_equal(got[:, :512].numpy(), codes)
        np.testing.assert_array_equal(got[:, 512:528].contiguous().view(torch.float32).numpy(),
                                      scales)
        tail = got[:, 528:656].contiguous().view(torch.bfloat16)
    else:
        assert torch.equal(got[:, :512], x[:, :512])
        tail = got[:, 512:576]
    _check_turned(tail.double(), x[:, 512:].double(), cos, sin, halves, U_BF16)


def _check_turned(got, x, cos, sin, halves, u):
    if cos is None:
        assert torch.equal(got, x)
        return
    ref = pagedlib.rotate(x, cos, sin, halves)
    size = pagedlib.rotate(x.abs(), cos.abs(), -sin.abs(), halves).abs() + \
        pagedlib.rotate(x.abs(), cos.abs(), sin.abs(), halves).abs()
    assert ((got - ref).abs() <= u * ref.abs() + 4 * U_F32 * size + 1e-38).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxf4"])
@pytest.mark.parametrize("kdt", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows,page,kvh,kh,turn", [(1, 16, False, False, True),
                                                   (5, 64, True, False, True),
                                                   (130, 32, False, True, True),
                                                   (63, 128, True, True, False)])
def test_cache_append(kind, kdt, rows, page, kvh, kh, turn):
    g = _gen(rows + page)
    pages = -(-rows // page) + 2
    kv = torch.randn(rows, 592, generator=g).bfloat16()
    kv[:, :512] *= torch.exp2(torch.randint(-6, 7, (rows, 16, 1), generator=g)).expand(
        rows, 16, 32).reshape(rows, 512)
    k = torch.randn(rows, 132, generator=g).bfloat16()
    table = ic.rope_table(5000, device=DEV)
    pos = torch.randint(0, 5000, (rows,), generator=g, dtype=torch.int32)
    slots = torch.randperm(pages * page, generator=g)[:rows]
    kvc, kc, ks = _caches(kind, kdt, pages, page, pad=16)
    kv_d, k_d = kv.to(DEV), k.to(DEV)
    ic.ic_cache_append(slots.to(DEV), kv=kv_d[:, :576], kv_cache=kvc, kv_dtype=KINDS[kind],
                       k=k_d[:, :128], k_cache=kc, k_scale=ks, kv_halves=kvh, k_halves=kh,
                       **(dict(pos=pos.to(DEV), rope=table) if turn else {}))
    ic.ic_device_status()
    cs = table.cpu().double()[pos.long()] if turn else None
    cos, sin = (cs[:, :32], cs[:, 32:]) if turn else (None, None)
    kvc, kc = kvc.flatten(0, 1).cpu(), kc.flatten(0, 1).cpu()
    _check_latent(kvc[slots], kv[:, :576], kind, cos, sin, kvh)
    x = k[:, :128].double()
    if kdt == "bf16":
        got = kc[slots].double()
        _check_turned(got[:, :64], x[:, :64], cos, sin, kh, U_BF16)
        assert torch.equal(got[:, 64:], x[:, 64:])
    else:
        ks = ks.flatten().cpu().double()
        ref = x.clone()
        if turn:
            ref[:, :64] = pagedlib.rotate(x[:, :64], cos, sin, kh)
        size = 2 * x.abs().amax(1, keepdim=True)      # |a cos| + |b sin| of a row at most
        want = ref.abs().amax(1) / 448
        sc = ks[slots]
        assert ((sc - want).abs() <= 4 * U_F32 * (size[:, 0] / 448 + want)).all()
        val = kc[slots].view(torch.float8_e4m3fn).float().double()
        q = ref / sc[:, None]
        lim = torch.maximum(pagedlib.e4m3_half_step(q.clamp(-448, 448)),
                            pagedlib.e4m3_half_step(val))
        assert ((val - q).abs() <= lim * (1 + 1e-6) + 8 * U_F32 * size / sc[:, None]).all()
    # nothing else was written
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[slots] = False
    assert (kvc[rest] == 7).all() and (kvc[:, WIDTH[kind]:] == 7).all() and (kc[rest] == 7).all()
    if kdt == "e4m3":
        assert (ks[rest] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxf4"])
def test_cache_append_skips_padded_and_outside_tokens(kind):
    g = _gen(4)
    kv, k = torch.randn(9, 576, generator=g).bfloat16(), torch.randn(9, 128, generator=g).bfloat16()
    kvc, kc, ks = _caches(kind, "e4m3", 2, 16)
    slots = torch.tensor([3, -1, 31, 32, 1 << 40, -(1 << 40), 5, 6, 7])
    pos = torch.tensor([0, 1, 2, 3, 4, 5, 10, -1, 9], dtype=torch.int32)  # the table has 0..9
    ic.ic_cache_append(slots.to(DEV), kv=kv.to(DEV), kv_cache=kvc, kv_dtype=KINDS[kind],
                       k=k.to(DEV), k_cache=kc, k_scale=ks, pos=pos.to(DEV),
                       rope=ic.rope_table(10, device=DEV))
    ic.ic_device_status()
    changed = (ks.flatten() != 7).nonzero().flatten().tolist()
    assert changed == [3, 7, 31]
    kvc = kvc.flatten(0, 1)
    same = [i for i in range(32) if i not in changed]
    assert (kvc[same] == 7).all() and not (kvc[changed] == 7).all(1).any()


def test_cache_append_one_of_the_two_caches_and_no_tokens():
    kv, k = torch.randn(3, 576).bfloat16().to(DEV), torch.randn(3, 128).bfloat16().to(DEV)
    slots = torch.tensor([2, 0, 1], device=DEV)
    kvc, kc, _ = _caches("bf16", "bf16", 1, 16)
    ic.ic_cache_append(slots, k=k, k_cache=kc)
    assert torch.equal(kc[0, slots], k) and (kvc == 7).all()
    ic.ic_cache_append(slots, kv=kv, kv_cache=kvc)
    assert torch.equal(kvc[0, slots], kv)
    ic.ic_cache_append(slots[:0], kv=kv[:0], kv_cache=kvc)
    ic.ic_device_status()


def test_cache_append_e4m3_equals_the_quantisers_bit_for_bit():
    """Rows of every magnitude that bf16 has, subnormal ones included, with values down to
    2^-24 of the largest: the codes and scales of ic_quant_e4m3_rows and ic_pack_kv_e4m3."""
    g = _gen(21)
    rows = 262
    top = torch.arange(-134, 128).double()[:, None]
    sign = torch.randint(0, 2, (rows, 704), generator=g) * 2 - 1
    x = sign * (1 + torch.rand(rows, 704, generator=g).double()) * \
        2.0 ** (top - torch.randint(0, 25, (rows, 704), generator=g))
    x = x.clamp(-3.3e38, 3.3e38).bfloat16().to(DEV)
    k, kv = x[:, :128].contiguous(), x[:, 128:].contiguous()
    kvc = torch.zeros(rows, 656, dtype=torch.uint8, device=DEV)
    kc = torch.zeros(rows, 128, dtype=torch.uint8, device=DEV)
    ks = torch.zeros(rows, device=DEV)
    ic.ic_cache_append(torch.arange(rows, device=DEV), kv=kv, kv_cache=kvc, kv_dtype=ic.IC_E4M3,
                       k=k, k_cache=kc, k_scale=ks)
    codes, scales = ic.ic_quant_e4m3_rows(k)
    packed = ic.ic_pack_kv_e4m3(kv)
    ic.ic_device_status()
    assert torch.equal(kc, codes) and torch.equal(ks, scales.flatten())
    assert torch.equal(kvc, packed.view(rows, 656))


def test_cache_append_mxf4_edge_blocks_bit_exact():
    """Zeros, subnormals, the largest bf16, infinities and NaN, every tie of the format, and
    magnitudes on both sides of 1.5 times a power of two."""
    x = torch.zeros(24, 576).bfloat16()
    ties = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0,
                         6.0, 5.5])
    for r in range(8):
        s = 2.0 ** (r * 10 - 40)
        x[r, :16] = (ties * s).bfloat16()
        x[r, 16:32] = (-ties * s).bfloat16()
        x[r, 32] = 1.5 * s
        x[r, 64] = 1.5078125 * s
        x[r, 96] = 1.9921875 * s
        x[r, 128] = -s
    x[8, 0] = torch.finfo(torch.bfloat16).max
    x[8, 32] = torch.finfo(torch.bfloat16).tiny
    x[8, 64] = torch.finfo(torch.bfloat16).tiny / 4      # subnormals
    x[8, 96] = -torch.finfo(torch.bfloat16).tiny / 128
    x[9, 5] = math.inf
    x[9, 40] = -math.inf
    x[10, 70] = math.nan
    x[11, :512] = -0.0
    g = _gen(9)
    x[12:] = (torch.randn(12, 576, generator=g) *
              torch.exp2(torch.randint(-100, 100, (12, 576), generator=g))).bfloat16()
    cache = torch.zeros(24, 400, dtype=torch.uint8, device=DEV)
    ic.ic_cache_append(torch.arange(24, device=DEV), kv=x.to(DEV), kv_cache=cache,
                       kv_dtype=ic.IC_MXF4)
    ic.ic_device_status()
    np.testing.assert_array_equal(cache.cpu().numpy(), pagedlib.pack_mxf4(x.double().numpy()))


# ------------------------------------------------------------------------------- indexer
def _index_inputs(lens, page, fp8, seed, fill=-1):
    g = _gen(seed)
    B = len(lens)
    table, pages = pagedlib.shuffled_table(lens, page, 2, g, fill)
    q = (torch.randn(B, 64, 128, generator=g) / 128 ** 0.5).bfloat16()
    k = (torch.randn(pages * page, 128, generator=g) / 128 ** 0.5).bfloat16()
    w = torch.rand(B, 64, generator=g) / 8
    used = torch.zeros(pages * page, dtype=torch.bool)
    for b, n in enumerate(lens):
        used[pagedlib.paged_rows(table, b, torch.arange(n), page)] = True
    k[~used] = math.nan                                   # rows of no token
    d = dict(q=q.to(DEV), k=k.to(DEV), w=w.to(DEV), q_scale=None, k_scale=None)
    if fp8:
        d["q"], d["q_scale"] = ic.ic_quant_e4m3_rows(d["q"])
        d["k"], d["k_scale"] = ic.ic_quant_e4m3_rows(d["k"])
        d["k_scale"][~used.to(DEV)] = math.nan
    return d, table


def _index_values(d):
    """(q, k) in 64 bits."""
    if d["q_scale"] is None:
        return d["q"].double(), d["k"].double()
    f8 = torch.float8_e4m3fn
    return (d["q"].view(f8).float().double() * d["q_scale"].double()[..., None],
            d["k"].view(f8).float().double() * d["k_scale"].double()[:, None])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
def test_indexer_paged(fp8, page):
    lens = [0, 1, 127, 128, 129, 0, 0, 1000, 2500, 16, 15, 17, 0]
    d, table = _index_inputs(lens, page, fp8, page)
    max_len = 2500
    scores = torch.full((len(lens), max_len + 4), 9.0, device=DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ic.ic_indexer_scores_paged(d["q"], d["k"], d["w"], table.to(DEV), sl, page_size=page,
                               scores=scores[:, :max_len], q_scale=d["q_scale"],
                               k_scale=d["k_scale"])
    ic.ic_device_status()
    q, k = _index_values(d)
    for b, n in enumerate(lens):
        assert (scores[b, n:] == 9.0).all()
        if n == 0:
            continue
        rows = pagedlib.paged_rows(table, b, torch.arange(n), page).to(DEV)
        w = d["w"][b].double()
        ref = w @ (q[b] @ k[rows].T).clamp(min=0)
        # a dot product of 128 terms and a sum of 64, one fp32 step each
        size = w @ (q[b].abs() @ k[rows].abs().T)
        assert ((scores[b, :n].double() - ref).abs() <= 200 * 2 * U_F32 * size).all()
        # the same bits as over a contiguous copy of the keys
        ks = None if d["k_scale"] is None else d["k_scale"][rows].contiguous()
        qs = None if d["q_scale"] is None else d["q_scale"][b:b + 1]
        dense = ic.ic_indexer_scores(d["q"][b:b + 1], d["k"][rows].contiguous(), d["w"][b:b + 1],
                                     pos0=n - 1, q_scale=qs, k_scale=ks)
        assert torch.equal(dense[0], scores[b, :n])


def test_indexer_paged_clamps_lengths_and_survives_bad_pages():
    lens = [300, 200]
    d, table = _index_inputs(lens, 64, True, 3)
    table[0, 2] = -5                                     # tokens 128..191 of sequence 0
    table[1, 1] = 1 << 20
    sl = torch.tensor([1 << 30, -4], dtype=torch.int32, device=DEV)
    scores = torch.full((2, 260), 9.0, device=DEV)
    ic.ic_indexer_scores_paged(d["q"], d["k"], d["w"], table.to(DEV), sl, page_size=64,
                               scores=scores, q_scale=d["q_scale"], k_scale=d["k_scale"])
    torch.cuda.synchronize()
    assert (scores[0, 128:192] == 0).all() and (scores[0, :128] != 9).all()
    assert (scores[0, 192:256] != 9).all() and (scores[0, 256:] != 9).all()
    assert (scores[1] == 9).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_indexer_paged_many_sequences(fp8):
    """More sequences than CTAs, and one long row: shares cut inside and across sequences."""
    lens = [(37 * i) % 301 for i in range(400)] + [40000]
    d, table = _index_inputs(lens, 32, fp8, 8)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    scores = ic.ic_indexer_scores_paged(d["q"], d["k"], d["w"], table.to(DEV), sl, page_size=32,
                                        q_scale=d["q_scale"], k_scale=d["k_scale"])
    ic.ic_device_status()
    q, k = _index_values(d)
    for b in list(range(0, 400, 13)) + [400]:
        n = lens[b]
        rows = pagedlib.paged_rows(table, b, torch.arange(n), 32).to(DEV)
        w = d["w"][b].double()
        ref = w @ (q[b] @ k[rows].T).clamp(min=0)
        size = w @ (q[b].abs() @ k[rows].abs().T)
        assert ((scores[b, :n].double() - ref).abs() <= 200 * 2 * U_F32 * size).all()


def test_all_sequences_empty():
    d, table = _index_inputs([5, 5], 16, True, 1)
    sl = torch.zeros(2, dtype=torch.int32, device=DEV)
    scores = torch.full((2, 16), 9.0, device=DEV)
    ic.ic_indexer_scores_paged(d["q"], d["k"], d["w"], table.to(DEV), sl, page_size=16,
                               scores=scores, q_scale=d["q_scale"], k_scale=d["k_scale"])
    idx = ic.ic_topk_varlen(scores, 8, sl)
    q = torch.randn(2, 1, 16, 576, device=DEV).bfloat16()
    kv = torch.full((32, 576), math.nan, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(2, 1, 16, device=DEV)
    out = ic.ic_sparse_attn_paged(q, kv, idx[:, None], table.to(DEV), sl, 0.04, page_size=16,
                                  lse=lse)
    ic.ic_device_status()
    assert (scores == 9).all() and (idx == -1).all()
    assert (out == 0).all() and torch.isneginf(lse).all()


# ------------------------------------------------------------------------------- attention
def _latent_pool(rows, kind, g):
    """(cache [rows, width] on the GPU, its values in 64 bits)."""
    x = (torch.randn(rows, 576, generator=g) *
         (0.5 + torch.rand(576, generator=g))).bfloat16()
    if kind == "bf16":
        c = x.to(DEV)
    else:
        c = torch.zeros(rows, WIDTH[kind], dtype=torch.uint8, device=DEV)
        ic.ic_cache_append(torch.arange(rows, device=DEV), kv=x.to(DEV), kv_cache=c,
                           kv_dtype=KINDS[kind])
    return c, pagedlib.unpack(c, kind)


def _check_attn(q, idx, lens, table, page, values, scale, out, lse):
    B, R = idx.shape[:2]
    for b in range(B):
        for r in range(R):
            t = idx[b, r].long()
            t = t[(t >= 0) & (t < lens[b])]
            kv = values[pagedlib.paged_rows(table, b, t, page).to(DEV)]
            o, l, spread, zsize = pagedlib.attention(q[b, r].double(), kv, scale)
            if t.numel() == 0:
                assert (out[b, r] == 0).all()
                assert lse is None or torch.isneginf(lse[b, r]).all()
                continue
            # logits: 576 products and sums, one fp32 step each, and the scaling; their
            # error acts on the probabilities, which round to bf16, as the output does
            dz = (576 + 4) * 2 * U_F32 * zsize
            lim = (U_BF16 + 2 * dz + 1e-5)[:, None] * spread + U_BF16 * o.abs()
            assert ((out[b, r].double() - o).abs() <= lim * (1 + U_BF16)).all(), (b, r)
            if lse is not None:
                assert ((lse[b, r].double() - l).abs() <= dz + 1e-5 + 4 * U_F32 * l.abs()).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxf4"])
@pytest.mark.parametrize("page,R,k,lens", [
    (64, 1, 2048, [3000, 2500]), (16, 1, 33, [50, 0, 1, 33, 700]), (32, 3, 100, [400, 90]),
    (128, 1, 1, [5]), (64, 7, 257, [1000, 0, 300]), (1024, 2, 31, [64, 2000])])
def test_attn_paged(kind, page, R, k, lens):
    g = _gen(page + R + k)
    B = len(lens)
    table, pages = pagedlib.shuffled_table(lens, page, 2, g)
    cache, values = _latent_pool(pages * page, kind, g)
    idx = torch.full((B, R, k), -1, dtype=torch.int32)
    for b in range(B):
        for r in range(R):
            m = min(k, lens[b])
            idx[b, r, :m] = torch.randperm(max(lens[b], 1), generator=g)[:m].int()
            if r == 1 and m > 3:                     # holes and entries past the sequence
                idx[b, r, 1] = -1
                idx[b, r, 2] = lens[b] + 3
    q = torch.randn(B, R, 16, 576, generator=g).bfloat16().to(DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    lse = torch.empty(B, R, 16, device=DEV)
    scale = 576 ** -0.5
    ws = torch.full((ic.ic_attn_workspace_size(B, R, 16, 512, k) // 4 + 4,), math.nan, device=DEV)
    args = (q, cache, idx.to(DEV), table.to(DEV), sl, scale)
    kw = dict(page_size=page, kv_dtype=KINDS[kind])
    out = ic.ic_sparse_attn_paged(*args, lse=lse, workspace=ws, **kw)
    ic.ic_device_status()
    _check_attn(q, idx, lens, table, page, values, scale, out, lse)
    whole = ic.ic_sparse_attn_paged(*args, **kw)         # no workspace: one CTA per query
    ic.ic_device_status()
    _check_attn(q, idx, lens, table, page, values, scale, whole, None)
    again = ic.ic_sparse_attn_paged(*args, workspace=ws, **kw)
    assert torch.equal(out, again)


def test_attn_paged_of_no_queries():
    pool = torch.zeros(4, 16, 576, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    lens = torch.ones(2, dtype=torch.int32, device=DEV)
    out = ic.ic_sparse_attn_paged(torch.empty(2, 0, 16, 576, dtype=torch.bfloat16, device=DEV), pool,
                                  torch.empty(2, 0, 8, dtype=torch.int32, device=DEV), table, lens,
                                  1.0, page_size=16)
    assert out.shape == (2, 0, 16, 512)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxf4"])
def test_attn_paged_of_many_queries(kind):
    """More queries than the split takes (600 > 4 per SM): persistent CTAs."""
    g = _gen(6)
    lens, page, R, k = [900, 1300], 64, 300, 70
    table, pages = pagedlib.shuffled_table(lens, page, 0, g)
    cache, values = _latent_pool(pages * page, kind, g)
    idx = torch.stack([torch.stack([torch.randperm(n - R + r + 1, generator=g)[:k].sort().values
                                    for r in range(R)]) for n in lens]).int()
    idx[0, 5] = -1
    idx[1, 7, 40:] = -1
    q = torch.randn(2, R, 16, 576, generator=g).bfloat16().to(DEV)
    lse = torch.empty(2, R, 16, device=DEV)
    out = ic.ic_sparse_attn_paged(q, cache, idx.to(DEV), table.to(DEV),
                                  torch.tensor(lens, dtype=torch.int32, device=DEV), 0.05,
                                  page_size=page, kv_dtype=KINDS[kind], lse=lse)
    ic.ic_device_status()
    _check_attn(q, idx, lens, table, page, values, 0.05, out, lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxf4"])
def test_attn_paged_non_finite_rows_stay_with_their_query(kind):
    """Query 0 selects rows of infinities and NaN; the others (fewer entries, so that tiles
    keep places without a row) must not see them."""
    g = _gen(12)
    lens, page, R, k = [200], 16, 700, 64
    table, pages = pagedlib.shuffled_table(lens, page, 0, g)
    x = torch.randn(pages * page, 576, generator=g).bfloat16()
    bad = pagedlib.paged_rows(table, 0, torch.arange(0, 64), page)
    x[bad[::2]] = math.inf
    x[bad[1::2]] = math.nan
    cache = x.to(DEV)
    if kind != "bf16":
        cache = torch.zeros(pages * page, WIDTH[kind], dtype=torch.uint8, device=DEV)
        ic.ic_cache_append(torch.arange(pages * page, device=DEV), kv=x.to(DEV), kv_cache=cache,
                           kv_dtype=KINDS[kind])
    values = pagedlib.unpack(cache, kind)
    idx = torch.full((1, R, k), -1, dtype=torch.int32)
    idx[0, 0::3] = torch.arange(64, dtype=torch.int32)   # the bad rows, in many queries
    for r in range(R):
        if r % 3:
            m = r % 40
            idx[0, r, :m] = (64 + torch.randperm(136, generator=g)[:m]).int()
    q = torch.randn(1, R, 16, 576, generator=g).bfloat16().to(DEV)
    out = ic.ic_sparse_attn_paged(q, cache, idx.to(DEV), table.to(DEV),
                                  torch.tensor(lens, dtype=torch.int32, device=DEV), 0.04,
                                  page_size=page, kv_dtype=KINDS[kind])
    ic.ic_device_status()
    good = [r for r in range(R) if r % 3]
    assert torch.isfinite(out[0, good]).all() and torch.isnan(out[0, 0]).all()
    _check_attn(q[:, good], idx[:, good], lens, table, page, values, 0.04, out[:, good], None)


def test_attn_paged_mxf4_scales_of_every_size():
    """Rows and blocks whose scales span the format: each query holds one size only."""
    g = _gen(13)
    n, page = 64, 64
    x = torch.randn(n, 576, generator=g)
    x[:32, :512] *= 2.0 ** -100
    x[32:, :512] *= 2.0 ** 100
    x[:, 512:] *= 0.5
    cache = torch.zeros(n, 400, dtype=torch.uint8, device=DEV)
    ic.ic_cache_append(torch.arange(n, device=DEV), kv=x.bfloat16().to(DEV), kv_cache=cache,
                       kv_dtype=ic.IC_MXF4)
    values = pagedlib.unpack(cache, "mxf4")
    idx = torch.arange(64, dtype=torch.int32).view(1, 2, 32)
    q = torch.randn(1, 2, 16, 576, generator=g)
    q[0, 1, :, :512] *= 2.0 ** -100
    q = q.bfloat16().to(DEV)
    table = torch.zeros(1, 1, dtype=torch.int32)
    out = ic.ic_sparse_attn_paged(q, cache, idx.to(DEV), table.to(DEV),
                                  torch.tensor([n], dtype=torch.int32, device=DEV), 0.04,
                                  page_size=page, kv_dtype=ic.IC_MXF4)
    ic.ic_device_status()
    _check_attn(q, idx, [n], table, page, values, 0.04, out, None)


def test_attn_paged_repeated_entries_count_twice_and_bad_pages_are_skipped():
    g = _gen(14)
    lens, page = [100], 16
    table, pages = pagedlib.shuffled_table(lens, page, 0, g)
    cache, values = _latent_pool(pages * page, "mxf4", g)
    idx = torch.tensor([[[5, 5, 7, 40, 41, 7, 99]]], dtype=torch.int32)
    q = torch.randn(1, 1, 16, 576, generator=g).bfloat16().to(DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = ic.ic_sparse_attn_paged(q, cache, idx.to(DEV), table.to(DEV), sl, 0.04, page_size=page,
                                  kv_dtype=ic.IC_MXF4)
    ic.ic_device_status()
    _check_attn(q, idx, lens, table, page, values, 0.04, out, None)
    broken = table.clone()
    broken[0, 2] = 1 << 30                               # tokens 32..47: 40 and 41
    out = ic.ic_sparse_attn_paged(q, cache, idx.to(DEV), broken.to(DEV), sl, 0.04, page_size=page,
                                  kv_dtype=ic.IC_MXF4)
    torch.cuda.synchronize()
    keep = idx.clone()
    keep[0, 0, 3:5] = -1
    _check_attn(q, keep, lens, table, page, values, 0.04, out, None)


@pytest.mark.parametrize("kind", ["bf16"])  # the packed rows have a kernel of their own
def test_attn_paged_equals_the_contiguous_call(kind):
    g = _gen(15)
    page, n, k = 64, 2048, 500
    cache, _ = _latent_pool(n, kind, g)
    idx = torch.stack([torch.randperm(n, generator=g)[:k].sort().values for _ in range(3)]).int()
    q = torch.randn(1, 3, 16, 576, generator=g).bfloat16().to(DEV)
    ws = torch.empty(ic.ic_attn_workspace_size(1, 3, 16, 512, k), dtype=torch.uint8, device=DEV)
    dense = ic.ic_sparse_attn(q, cache[None], idx[None].to(DEV), 0.04, workspace=ws)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV)[None]
    got = ic.ic_sparse_attn_paged(q, cache, idx[None].to(DEV), table,
                                  torch.tensor([n], dtype=torch.int32, device=DEV), 0.04,
                                  page_size=page, kv_dtype=KINDS[kind], workspace=ws)
    ic.ic_device_status()
    assert torch.equal(dense, got)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxf4"])
def test_attn_paged_loose_alignment_and_wide_tables(kind):
    """Index lists and outputs at 4-byte addresses, a workspace that the merge cannot use, a
    cache with longer rows, a block table and lengths inside larger tensors."""
    g = _gen(21)
    lens, page, k = [700, 333], 32, 256
    table, pages = pagedlib.shuffled_table(lens, page, 0, g)
    cache, values = _latent_pool(pages * page, kind, g)
    pad = 8 if kind == "bf16" else 16
    wide = torch.zeros(pages, page, cache.shape[1] + pad, dtype=cache.dtype, device=DEV)
    wide[..., :cache.shape[1]] = cache.view(pages, page, -1)
    idx = torch.stack([torch.randperm(n, generator=g)[:k].sort().values for n in lens]).int()
    flat = torch.empty(2 * k + 1, dtype=torch.int32, device=DEV)
    loose = flat[1:].view(2, 1, k)
    loose.copy_(idx[:, None])
    big = torch.full((2, 40), 1 << 28, dtype=torch.int32, device=DEV)
    big[:, 3:3 + table.shape[1]] = table.to(DEV)
    sl = torch.tensor([9] + lens, dtype=torch.int32, device=DEV)[1:]
    q = torch.randn(2, 1, 16, 576, generator=g).bfloat16().to(DEV)
    buf = torch.empty(2 * 16 * 512 + 2, dtype=torch.bfloat16, device=DEV)
    out = buf[2:].view(2, 1, 16, 512)
    lse = torch.empty(2, 1, 16, device=DEV)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)[4:]
    for w in (None, ws):
        out.fill_(0)
        got = ic.ic_sparse_attn_paged(q, wide[..., :cache.shape[1]], loose,
                                      big[:, 3:3 + table.shape[1]], sl, 0.04, page_size=page,
                                      kv_dtype=KINDS[kind], out=out, lse=lse, workspace=w)
        ic.ic_device_status()
        assert got is out
        _check_attn(q, idx[:, None], lens, table, page, values, 0.04, out, lse)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxf4"])
def test_attn_paged_many_empty_and_tiny_queries(kind):
    """Queries of 0, 1, 31..33 and 64..65 entries one after another in every CTA, with holes
    that leave a first tile without entries."""
    g = _gen(22)
    lens, page, R, k = [128], 16, 1500, 96
    table, pages = pagedlib.shuffled_table(lens, page, 0, g)
    cache, values = _latent_pool(pages * page, kind, g)
    idx = torch.full((1, R, k), -1, dtype=torch.int32)
    sizes = [0, 1, 31, 32, 33, 64, 65, 96, 0, 0, 5]
    for r in range(R):
        m = sizes[r % len(sizes)]
        idx[0, r, :m] = torch.randperm(128, generator=g)[:m].int()
        if r % 7 == 3:
            idx[0, r, :40] = -1
    q = torch.randn(1, R, 16, 576, generator=g).bfloat16().to(DEV)
    lse = torch.empty(1, R, 16, device=DEV)
    out = ic.ic_sparse_attn_paged(q, cache, idx.to(DEV), table.to(DEV),
                                  torch.tensor(lens, dtype=torch.int32, device=DEV), 0.05,
                                  page_size=page, kv_dtype=KINDS[kind], lse=lse)
    ic.ic_device_status()
    _check_attn(q, idx, lens, table, page, values, 0.05, out, lse)


@pytest.mark.parametrize("kind", ["e4m3", "mxf4"])
def test_attn_paged_rising_scores(kind):
    """Scores that grow along the list, so that the softmax's reference point has to follow,
    in small steps (within its slack) and in large ones; and falling ones."""
    g = _gen(23)
    n, page, k = 512, 64, 512
    x = torch.zeros(n, 576)
    x[:, :512] = torch.randn(n, 512, generator=g) * 0.1
    x[:, 512] = torch.arange(n) / 8.0                    # the score's trend, in a bf16 dim
    cache = torch.zeros(n, WIDTH[kind], dtype=torch.uint8, device=DEV)
    ic.ic_cache_append(torch.arange(n, device=DEV), kv=x.bfloat16().to(DEV), kv_cache=cache,
                       kv_dtype=KINDS[kind])
    values = pagedlib.unpack(cache, kind)
    q = torch.randn(1, 4, 16, 576, generator=g)
    q[..., 512:] = 0
    for r, slope in enumerate((0.25, 4.0, 200.0, 1000.0)):
        q[0, r, :, 512] = slope
    q = q.bfloat16().to(DEV)
    table = torch.arange(n // page, dtype=torch.int32)[None]
    sl = torch.tensor([n], dtype=torch.int32, device=DEV)
    for order in (torch.arange(n), torch.arange(n - 1, -1, -1)):
        idx = order.int().expand(1, 4, n).contiguous()
        lse = torch.empty(1, 4, 16, device=DEV)
        out = ic.ic_sparse_attn_paged(q, cache, idx.to(DEV), table.to(DEV), sl, 0.05,
                                      page_size=page, kv_dtype=KINDS[kind], lse=lse)
        ic.ic_device_status()
        _check_attn(q, idx, [n], table, page, values, 0.05, out, lse)


def test_paged_offsets_past_32_bits():
    """Pages at the far end of pools of more than 2^32 bytes."""
    page, n = 64, 300
    pages = (1 << 32) // (128 * page) + 100
    g = _gen(16)
    k = torch.empty(pages * page, 128, dtype=torch.uint8, device=DEV)
    ks = torch.empty(pages * page, device=DEV)
    kv = torch.empty(pages * page, 400, dtype=torch.uint8, device=DEV)
    table = torch.tensor([[pages - 1, 3, pages - 3, pages - 2, pages - 9]], dtype=torch.int32)
    rows = pagedlib.paged_rows(table, 0, torch.arange(n), page).to(DEV)
    x, y = torch.randn(n, 576, generator=g).bfloat16(), torch.randn(n, 128, generator=g).bfloat16()
    ic.ic_cache_append(rows, kv=x.to(DEV), kv_cache=kv, kv_dtype=ic.IC_MXF4, k=y.to(DEV),
                       k_cache=k, k_scale=ks)
    small, small_s = ic.ic_quant_e4m3_rows(y.to(DEV))
    assert torch.equal(k[rows], small) and torch.equal(ks[rows], small_s)
    q8, qs = ic.ic_quant_e4m3_rows(torch.randn(1, 64, 128, generator=g).bfloat16().to(DEV))
    w = torch.rand(1, 64, generator=g).to(DEV)
    sl = torch.tensor([n], dtype=torch.int32, device=DEV)
    got = ic.ic_indexer_scores_paged(q8, k, w, table.to(DEV), sl, page_size=page, q_scale=qs,
                                     k_scale=ks)
    dense = ic.ic_indexer_scores(q8, small, w, pos0=n - 1, q_scale=qs, k_scale=small_s)
    assert torch.equal(got[0, :n], dense[0])
    idx = torch.randperm(n, generator=g)[None, None].int()
    q = torch.randn(1, 1, 16, 576, generator=g).bfloat16().to(DEV)
    out = ic.ic_sparse_attn_paged(q, kv, idx.to(DEV), table.to(DEV), sl, 0.04, page_size=page,
                                  kv_dtype=ic.IC_MXF4)
    ic.ic_device_status()
    values = torch.zeros(n, 576, dtype=torch.float64, device=DEV)
    values[:] = pagedlib.unpack(kv[rows], "mxf4")
    flat = torch.arange(5, dtype=torch.int32)[None]
    pool = torch.zeros(5 * page, 576, dtype=torch.float64, device=DEV)
    pool[:n] = values
    _check_attn(q, idx, [n], flat, page, pool, 0.04, out, None)


# ------------------------------------------------------------------------------- together
class _Serving:
    """A small paged serving state: caches of two layers (F, S), filled through the append."""

    def __init__(self, kind, kdt, lens, page, k, cap, seed):
        g = self.g = _gen(seed)
        self.kind, self.kdt, self.page, self.k, self.cap = kind, kdt, page, k, cap
        self.B, self.lens = len(lens), list(lens)
        self.table, self.pages = pagedlib.shuffled_table([cap] * self.B, page, 3, g)
        self.dtable = self.table.to(DEV)
        self.sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.rope = ic.rope_table(cap, device=DEV)
        self.pools = [_caches(kind, kdt, self.pages, page) for _ in range(2)]
        for layer in range(2):
            slots, pos = [], []
            for b, n in enumerate(lens):
                t = torch.arange(n)
                slots.append(pagedlib.paged_rows(self.table, b, t, page))
                pos.append(t)
            self.append(layer, torch.cat(slots), torch.cat(pos))
        self.t_cache = torch.full((self.B, k), -7, dtype=torch.int32, device=DEV)
        self.layers = []
        for layer in range(2):
            kvc, kc, ks = self.pools[layer]
            q_idx = (torch.randn(self.B, 1, 64, 128, generator=g) / 11).bfloat16().to(DEV)
            e = dict(w=torch.rand(self.B, 1, 64, generator=g).to(DEV) / 8, k_idx=kc, k_scale=ks,
                     kv=kvc, q=torch.randn(self.B, 1, 16, 576, generator=g).bfloat16().to(DEV),
                     out=torch.zeros(self.B, 1, 16, 512, dtype=torch.bfloat16, device=DEV),
                     lse=torch.zeros(self.B, 1, 16, device=DEV))
            e["q_idx"], e["q_scale"] = (q_idx, None) if kdt == "bf16" else \
                ic.ic_quant_e4m3_rows(q_idx)
            self.layers.append(e)
        self.desc = ic.make_desc(L=cap, k=k, H=64, D=128, heads=16, dk=576, dv=512,
                                 idx_dtype=KINDS[kdt], attn_dtype=KINDS[kind], scale=576 ** -0.5,
                                 ld_kv=WIDTH[kind], batch=self.B, decode=True)
        self.paging = ic.make_paging(self.dtable, self.sl, page, self.pages)
        self.ws = torch.empty(ic.ic_stack_workspace_size(self.desc) // 4 + 4, device=DEV)

    def append(self, layer, slots, pos):
        kvc, kc, ks = self.pools[layer]
        n = slots.numel()
        self.new_kv = torch.randn(n, 576, generator=self.g).bfloat16().to(DEV)
        self.new_k = torch.randn(n, 128, generator=self.g).bfloat16().to(DEV)
        ic.ic_cache_append(slots.to(DEV), kv=self.new_kv, kv_cache=kvc,
                           kv_dtype=KINDS[self.kind], k=self.new_k, k_cache=kc, k_scale=ks,
                           pos=pos.int().to(DEV), rope=self.rope)

    def step(self, **kw):
        ic.ic_decode_step_paged("F,S", self.desc, self.paging, self.layers, self.t_cache,
                                kw.pop("ws", self.ws), **kw)

    def check(self):
        """T against the plain top-k of the paged scores, the outputs against 64 bits."""
        e = self.layers[0]
        kc, ks = self.pools[0][1:]
        d = dict(q=e["q_idx"][:, 0], k=kc.flatten(0, 1), q_scale=None, k_scale=None)
        if ks is not None:
            d.update(q_scale=e["q_scale"][:, 0], k_scale=ks.flatten())
        q, k = _index_values(d)
        T = self.t_cache.cpu()
        for b, n in enumerate(self.lens):
            m = min(n, self.k)
            t = T[b, :m].long()
            assert (T[b, m:] == -1).all() and (t.diff() > 0).all()
            assert m == 0 or (t[0] >= 0 and t[-1] < n)
            if m == 0:
                continue
            rows = pagedlib.paged_rows(self.table, b, torch.arange(n), self.page).to(DEV)
            w = e["w"][b, 0].double()
            s = w @ (q[b] @ k[rows].T).clamp(min=0)
            size = (w @ (q[b].abs() @ k[rows].abs().T)).amax() * 200 * 2 * U_F32
            kth = s.topk(m).values[-1]
            picked = torch.zeros(n, dtype=torch.bool, device=DEV)
            picked[t.to(DEV)] = True
            assert (s[picked] >= kth - 2 * size).all() and (s[~picked] <= kth + 2 * size).all()
        for layer in range(2):
            e = self.layers[layer]
            values = pagedlib.unpack(self.pools[layer][0].flatten(0, 1), self.kind)
            _check_attn(e["q"], T[:, None], self.lens, self.table, self.page, values,
                        576 ** -0.5, e["out"], e["lse"])


@pytest.mark.parametrize("kind,kdt", [("mxf4", "e4m3"), ("e4m3", "e4m3"), ("bf16", "bf16"),
                                      ("mxf4", "bf16")])
def test_append_then_decode_step_ragged(kind, kdt):
    s = _Serving(kind, kdt, [700, 0, 1, 300, 64, 65, 1000], 64, 128, 1024, 31)
    s.step()
    ic.ic_device_status()
    s.check()
    first = [e["out"].clone() for e in s.layers] + [s.t_cache.clone()]
    # one score row at a time: the same bits
    s.step(ws=torch.empty(1024, device=DEV))
    ic.ic_device_status()
    assert torch.equal(first[2], s.t_cache)
    s.check()


def test_decode_step_paged_equals_the_contiguous_step():
    """Equal lengths, bf16 latents: T and outputs are those of ic_decode_step on copies."""
    n, B = 640, 5
    s = _Serving("bf16", "e4m3", [n] * B, 128, 200, n, 32)
    s.step()
    layers = []
    for layer, e in enumerate(s.layers):
        kvc, kc, ks = (p.flatten(0, 1) for p in s.pools[layer])
        rows = torch.stack([pagedlib.paged_rows(s.table, b, torch.arange(n), 128)
                            for b in range(B)]).to(DEV)
        layers.append(dict(e, k_idx=kc[rows].contiguous(), k_scale=ks[rows].contiguous(),
                           kv=kvc[rows].contiguous(), out=torch.zeros_like(e["out"])))
    t = torch.empty_like(s.t_cache)
    ic.ic_decode_step("F,S", s.desc, layers, t, s.ws)
    ic.ic_device_status()
    assert torch.equal(t, s.t_cache)
    for a, b in zip(s.layers, layers):
        assert torch.equal(a["out"], b["out"])


def test_append_and_decode_step_captured_and_replayed_as_sequences_grow():
    """One captured step (append, indexer, top-k, attention) replayed with the inputs, slots,
    lengths and a padded sequence updated in place."""
    B, cap, page = 4, 512, 32
    s = _Serving("mxf4", "e4m3", [100, 31, 500, 0], page, 64, cap, 33)
    slots = torch.full((B,), -1, dtype=torch.int64, device=DEV)
    pos = torch.zeros(B, dtype=torch.int32, device=DEV)
    kv = torch.zeros(2, B, 576, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(2, B, 128, dtype=torch.bfloat16, device=DEV)
    h = torch.zeros(B, 512, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    lat = torch.zeros(2, B, 576, dtype=torch.bfloat16, device=DEV)

    def step():
        for layer in range(2):
            kvc, kc, ks = s.pools[layer]
            lat[layer].copy_(kv[layer])
            ic.ic_rms_norm(kv[layer][:, :512], w, 1e-6, h=h, y=lat[layer][:, :512])
            ic.ic_cache_append(slots, kv=lat[layer], kv_cache=kvc, kv_dtype=ic.IC_MXF4,
                               k=k[layer], k_cache=kc, k_scale=ks, pos=pos, rope=s.rope)
        s.step()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        step()
    for it in range(3):
        live = [b for b in range(B) if b != 3 or it == 2]      # sequence 3 is padding at first
        for b in live:
            s.lens[b] += 1
        at = [int(pagedlib.paged_rows(s.table, b, torch.tensor([s.lens[b] - 1]), page))
              if b in live else -1 for b in range(B)]
        slots.copy_(torch.tensor(at))
        pos.copy_(torch.tensor([max(n - 1, 0) for n in s.lens], dtype=torch.int32))
        s.sl.copy_(torch.tensor(s.lens, dtype=torch.int32))
        kv.copy_(torch.randn(2, B, 576, generator=s.g))
        k.copy_(torch.randn(2, B, 128, generator=s.g))
        graph.replay()
        ic.ic_device_status()
        s.check()
        norm = lat.cpu()
        for layer in range(2):
            rows = s.pools[layer][0].flatten(0, 1).cpu()
            for b in live:
                cs = s.rope.cpu().double()[s.lens[b] - 1][None]
                _check_latent(rows[at[b]][None], norm[layer, b][None], "mxf4", cs[:, :32],
                              cs[:, 32:], False)
    del graph


def test_paged_calls_on_another_stream_and_of_two_graphs():
    """Two states, each on its own stream with its own workspace, at the same time."""
    a = _Serving("mxf4", "e4m3", [400, 900, 20], 64, 256, 1024, 41)
    b = _Serving("e4m3", "bf16", [1000, 10, 0, 500], 16, 100, 1024, 42)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.step(stream=sa)
        b.step(stream=sb)
    ic.ic_device_status(sa)
    ic.ic_device_status(sb)
    a.check()
    b.check()
    x = torch.randn(64, 512, device=DEV).bfloat16()
    w = torch.ones(512, device=DEV)
    torch.cuda.synchronize()
    y, _, _ = ic.ic_rms_norm(x, w, stream=sa)
    sa.synchronize()
    _check_norm(x, None, w, 1e-6, None, y, None, None)


def test_trace_names_the_new_launches():
    s = _Serving("mxf4", "e4m3", [400, 90], 64, 64, 512, 43)
    x = torch.randn(4, 512, device=DEV).bfloat16()
    ic.ic_trace_begin(64)
    ic.ic_rms_norm(x, torch.ones(512, device=DEV), y=torch.empty_like(x))
    s.append(0, torch.arange(4), torch.arange(4))
    s.step()
    n, got = ic.ic_trace_end(64)
    names = [g[0] for g in got]
    assert names[:4] == ["rms_norm", "cache_append", "indexer_tc_e4m3", "topk"]
    assert "attn_mla_kv4" in names and n == len(names)
