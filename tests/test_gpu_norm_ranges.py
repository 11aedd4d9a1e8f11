"""The norm where h * gamma leaves fp32's range although the result does not.

Bounds as in test_gpu_norm: 2^-8 for y's rounding to bf16 and 41 * 2^-24 for
the fp32 arithmetic; h, q equal to the oracle's."""
import numpy as np
import pytest
import torch

import oracle
import block_draft_synth as syn
from helpers import dev_bf16

pytestmark = pytest.mark.gpu

ARITH = 41 * 2.0 ** -24
bits = syn.f32_to_bf16_bits


def _rows(d, repeat):
    rng = np.random.default_rng(d)
    x = rng.standard_normal((6, d)).astype(np.float32)
    x[0] = 3e38                                         # times 1.2: beyond fp32
    x[1] = np.where(rng.random(d) < 0.5, -3e38, 2.5e38)
    x[2] *= 2.0 ** 100
    x[3] *= 2.0 ** 100
    x[3, 5] = 3e38
    x[4, 7] = -1e30                                     # one channel far above the others
    return bits(np.tile(x, (repeat, 1)))


@pytest.mark.parametrize("repeat", [1, 60])
@pytest.mark.parametrize("d", [264, 512, 2560, 8200])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 20, 2.0 ** 62, 2.0 ** -40])
def test_products_beyond_fp32(d, repeat, scale):
    import block_draft_selection_b200 as bds
    x = _rows(d, repeat)
    rng = np.random.default_rng(d + 1)
    gamma = 1 + 0.2 * rng.standard_normal(d)
    gamma[::3] *= -1
    g = bits((gamma * scale).astype(np.float32))
    y, _ = bds.dflash_rmsnorm(dev_bf16(x), dev_bf16(g))
    q, s, _ = bds.dflash_rmsnorm_i8(dev_bf16(x), dev_bf16(g))
    yr, _, _ = oracle.rmsnorm(x, g)
    got = y.float().cpu().numpy().astype(np.float64)
    bad = ~(np.abs(got - yr) <= (2.0 ** -8 + 2 * ARITH) * np.abs(yr) + 1e-37)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], yr[bad][:4])
    qr, sr, _ = oracle.rmsnorm_i8(x, g)
    got = s.cpu().numpy()
    bad = ~(np.abs(got - sr) <= ARITH * sr)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], sr[bad][:4])
    np.testing.assert_array_equal(q.cpu().numpy(), qr)


def test_residual_sum_beyond_fp32_products():
    """The same with a residual: h itself is what the sum rounds to."""
    import block_draft_selection_b200 as bds
    d = 1024
    x = _rows(d, 1)
    res = bits((np.random.default_rng(3).standard_normal((6, d)) * 1e30).astype(np.float32))
    g = bits(np.linspace(-2, 2, d).astype(np.float32))
    y, h = bds.dflash_rmsnorm(dev_bf16(x), dev_bf16(g), residual=dev_bf16(res))
    q, s, h2 = bds.dflash_rmsnorm_i8(dev_bf16(x), dev_bf16(g), residual=dev_bf16(res))
    yr, hr, _ = oracle.rmsnorm(x, g, res)
    for t in (h, h2):
        np.testing.assert_array_equal(t.double().cpu().numpy(), hr)
    assert (np.abs(y.double().cpu().numpy() - yr) <= (2.0 ** -8 + 2 * ARITH) * np.abs(yr) + 1e-37).all()
    qr, sr, _ = oracle.rmsnorm_i8(x, g, res)
    np.testing.assert_array_equal(q.cpu().numpy(), qr)
    assert (np.abs(s.cpu().numpy() - sr) <= ARITH * sr).all()


def test_infinities_stay_infinities():
    """A row with an infinity among values whose products overflow is still one with a NaN scale."""
    import block_draft_selection_b200 as bds
    x = torch.full((3, 512), 3e38, dtype=torch.bfloat16, device="cuda")
    x[1, 100] = float("inf")
    x[2, 100] = float("nan")
    g = torch.full((512,), 1.5, dtype=torch.bfloat16, device="cuda")
    q, s, _ = bds.dflash_rmsnorm_i8(x, g)
    y, _ = bds.dflash_rmsnorm(x, g)
    assert torch.isfinite(s[0]) and (q[0] == 127).all() and (y[0] == 1.5).all()
    assert torch.isnan(s[1:]).all() and not q[1:].any()
    assert torch.isnan(y[1, 100]) and not y[1, :100].any() and torch.isnan(y[2]).all()
