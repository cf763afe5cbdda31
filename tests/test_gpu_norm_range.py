"""RMS norm of rows at the ends of its range: millions of values, tiny and huge ones."""
import math

import pytest
import torch

from sparse_attention_indexer_sum_b200 import binding as ic

pytestmark = pytest.mark.gpu
DEV = "cuda"
U_F32 = 2.0 ** -24


# 2^24 + 1 values: a 32-bit sum of 65536 terms a thread would be off by 2^-9 and more
@pytest.mark.parametrize("n", [20001, 1 << 20, 3_000_001, (1 << 24) + 1])
@pytest.mark.parametrize("value", [1.0488088130950928, 0.7, 0.9999999403953552])
def test_long_rows_of_equal_values(n, value):
    x = torch.full((2, n), value, device=DEV)
    x[1] *= -3.0
    w = torch.full((n,), 1.5, device=DEV)
    y, _, _ = ic.ic_rms_norm(x, w, 0.0)
    ic.ic_device_status()
    # squares and runs of 16 of them (17 steps, halved by the root), the mean, the root (2
    # steps) and two products, whatever n is
    lim = (17 / 2 + 1 + 2 + 2) * U_F32 * 1.5
    assert (y[0].double() - 1.5).abs().max() <= lim
    assert (y[1].double() + 1.5).abs().max() <= lim


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("res", [False, True])
def test_long_random_rows(dt, res):
    g = torch.Generator(device=DEV).manual_seed(3)
    n = 5_000_003
    x = torch.randn(1, n, generator=g, device=DEV).to(dt)
    r = torch.randn(1, n, generator=g, device=DEV).to(dt) if res else None
    w = torch.rand(n, generator=g, device=DEV)
    y, _, _ = ic.ic_rms_norm(x.float(), w, 1e-6, residual=None if r is None else r.float())
    ic.ic_device_status()
    h = x.double() + (0 if r is None else r.double())
    gain = w.double() / (h.pow(2).mean() + 1e-6).sqrt()  # ref / h, also where h is 0
    ref = h * gain
    # as above, and the addition x + r
    mag = (x.double().abs() + (0 if r is None else r.double().abs())) * gain
    lim = (17 / 2 + 5) * U_F32 * ref.abs() + 2 * U_F32 * mag + 1e-37
    assert ((y.double() - ref).abs() <= lim).all()


@pytest.mark.parametrize("n", [8, 512, 509, 8200, 16384, 20001])
@pytest.mark.parametrize("dt,size", [(torch.float32, 2.0 ** -140), (torch.float32, 2.0 ** -126),
                                     (torch.float32, 2.0 ** -100), (torch.float32, 2.0 ** -72),
                                     (torch.float32, 2.0 ** -40), (torch.float32, 2.0 ** 50),
                                     (torch.bfloat16, 2.0 ** -120), (torch.bfloat16, 2.0 ** -70),
                                     (torch.bfloat16, 2.0 ** 50)])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-29])
def test_rows_of_every_size(n, dt, size, eps):
    """Small rows, whose squares vanish in 32 bits, with an eps that covers them and without;
    the scale of such a row may itself be no normal 32-bit number.  (Squares of 2^50 and rows
    of 20001 stay below the documented limit.)"""
    g = torch.Generator().manual_seed(n)
    x = ((torch.randn(3, n, generator=g).clamp(-6, 6) + 0.01).double() * size).to(dt).to(DEV)
    x[2] = 1.0                             # a row of ordinary size beside them
    w = (1 + 0.2 * torch.randn(n, generator=g)).to(DEV)
    h, y = torch.empty_like(x), torch.empty_like(x)
    codes = torch.empty(3, n, dtype=torch.uint8, device=DEV)
    scales = torch.empty(3, -(-n // 128), device=DEV)
    ic.ic_rms_norm(x, w, eps, h=h, y=y, codes=codes, scales=scales)
    ic.ic_device_status()
    assert torch.equal(h, x)
    xd = x.double()
    eps32 = float(torch.tensor(eps, dtype=torch.float32))   # as the call takes it
    ref = xd / (xd.pow(2).mean(-1, keepdim=True) + eps32).sqrt() * w.double()
    assert ref[:2].abs().amax() > 0.1 or eps > size ** 2 / 100
    # the sum (n / 256 + 11 terms at most in a chain, halved by the root), the root and the
    # products; a result below the normal numbers keeps half a step of the smallest
    rel = ((min(n, 16384) / 256 + 17) / 2 + 8) * U_F32
    u = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -149 if dt == torch.float32 else 2.0 ** -133
    assert ((y.double() - ref).abs() <= (u + rel * (1 + u)) * ref.abs() + tiny).all()
    m = -(-n // 128)
    pad = torch.nn.functional.pad(ref, (0, m * 128 - n)).unflatten(-1, (m, 128))
    want = pad.abs().amax(-1) / 448
    assert ((scales.double() - want).abs() <= (rel + 4 * U_F32) * want + 2.0 ** -148).all()


@pytest.mark.parametrize("n", [512, 509])
def test_zero_rows(n):
    x = torch.zeros(2, n, device=DEV)
    w = torch.ones(n, device=DEV)
    assert (ic.ic_rms_norm(x, w, 1e-6)[0] == 0).all()
    assert (ic.ic_rms_norm(x, w, 2.0 ** -149)[0] == 0).all()
    assert torch.isnan(ic.ic_rms_norm(x, w, 0.0)[0]).all()     # 0 / 0
    ic.ic_device_status()
