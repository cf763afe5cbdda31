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
