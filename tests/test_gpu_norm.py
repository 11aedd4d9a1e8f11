"""RMS norm (bf16 and int8 output) and row quantisation on the GPU against the
fp64 oracle.

h and q must equal the oracle's bit for bit: h is one rounding of a sum that
fp32 holds well enough for it, and q is decided exactly (see the kernel).
y: relative 2^-8 for its rounding to bf16 plus the fp32 arithmetic's: a sum of
squares of at most 32 terms in a row per thread, 5 shuffle levels and up to 32
warps added one after another (69 roundings, halved by the square root), then
the mean, the reciprocal square root (two units in the last place: 4 * 2^-24)
and two products -- 41 * 2^-24.  scale: the same 41, with a product and a
division in place of the two products."""
import numpy as np
import pytest
import torch

import oracle
import block_draft_synth as syn
from helpers import dev_bf16

pytestmark = pytest.mark.gpu

ARITH = 41 * 2.0 ** -24
bits = syn.f32_to_bf16_bits


def _np_bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def _inputs(M, d, seed, residual):
    rng = np.random.default_rng(seed)
    wide = np.where(rng.random(d) < 0.02, 16.0, 1.0)
    x = bits((rng.standard_normal((M, d)) * wide).astype(np.float32))
    res = bits((3 * rng.standard_normal((M, d)) * wide).astype(np.float32)) if residual else None
    g = bits((1 + 0.2 * rng.standard_normal(d)).astype(np.float32))
    return x, res, g


def _check(x, res, g, eps=1e-6):
    import block_draft_selection_b200 as bds
    dx, dg = dev_bf16(x), dev_bf16(g)
    dr = None if res is None else dev_bf16(res)
    y, h = bds.dflash_rmsnorm(dx, dg, residual=dr, eps=eps)
    q, scale, h2 = bds.dflash_rmsnorm_i8(dx, dg, residual=dr, eps=eps)
    torch.cuda.synchronize()
    yr, hr, r = oracle.rmsnorm(x, g, res, eps)
    if res is None:
        assert h is None and h2 is None
    else:
        for t in (h, h2):
            np.testing.assert_array_equal(syn.bf16_bits_to_f32(_np_bits(t)).astype(np.float64), hr)
    got = y.float().cpu().numpy().astype(np.float64)
    assert (np.abs(got - yr) <= (2.0 ** -8 + 2 * ARITH) * np.abs(yr) + 1e-37).all()
    qr, sr, _ = oracle.rmsnorm_i8(x, g, res, eps)
    np.testing.assert_array_equal(q.cpu().numpy(), qr)
    assert (np.abs(scale.cpu().numpy() - sr) <= ARITH * sr).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,d", [(1, 8), (1, 256), (3, 264), (8, 2560), (447, 4096), (5, 4104), (64, 5120), (2, 8192),
                                 (3, 8200), (2, 16384), (1, 32768), (1000, 40),
                                 (301, 256), (150, 264), (333, 512), (201, 520), (1001, 1024), (203, 1032),
                                 (5003, 8)])
def test_norm(M, d, residual):
    _check(*_inputs(M, d, M + d, residual))


@pytest.mark.parametrize("eps", [1e-20, 1e-5, 0.5])
def test_eps(eps):
    x, res, g = _inputs(7, 2560, 3, True)
    _check(x, res, g, eps)


@pytest.mark.parametrize("repeat", [1, 60])   # a CTA a row; more rows than SMs: a warp a row where d allows it
@pytest.mark.parametrize("d", [2560, 640])
def test_extreme_rows(d, repeat):
    """Rows of zeros, of values whose squares leave fp32, of tiny values, one
    value alone, negative gamma; the squares' sum is taken in fp64 where fp32
    overflows."""
    rng = np.random.default_rng(5)
    X = rng.standard_normal((7, d)).astype(np.float32)
    X[0] = 0
    X[1] *= 2.0 ** 80
    X[2] *= 2.0 ** -60
    X[3] = 0
    X[3, 234] = -7
    X[4] = 3e38
    X[5] = 127 * np.where(rng.random(d) < 0.5, 0.5, -1.5) / 2 ** 7
    X[5, 0] = 127
    g = 1 + 0.2 * rng.standard_normal(d)
    g[::3] *= -1
    for gamma in (g.astype(np.float32), np.ones(d, np.float32), np.full(d, 0.25, np.float32)):
        x = X.copy()
        if gamma[0] not in (1.0, 0.25):
            x[4] = 1e37         # 3e38 times gamma would leave fp32
        _check(bits(np.tile(x, (repeat, 1))), None, bits(gamma))


def test_non_finite_rows():
    """A NaN or an infinity poisons its own row's scale and no other row."""
    import block_draft_selection_b200 as bds
    d = 512
    x, _, g = _inputs(5, d, 9, False)
    clean = bds.dflash_rmsnorm_i8(dev_bf16(x), dev_bf16(g))
    v = dev_bf16(x)
    v[1, 17] = float("nan")
    v[3, 500] = float("-inf")
    q, scale, _ = bds.dflash_rmsnorm_i8(v, dev_bf16(g))
    q2, scale2 = bds.dflash_quant_i8(v)
    y, _ = bds.dflash_rmsnorm(v, dev_bf16(g))
    for s, k in ((scale, q), (scale2, q2)):
        assert torch.isnan(s[[1, 3]]).all() and not k[[1, 3]].any()
    for m in (0, 2, 4):
        assert torch.equal(q[m], clean[0][m]) and scale[m] == clean[1][m]
        assert torch.isfinite(y[m].float()).all()
    assert torch.isnan(y[1].float()).all()
    assert torch.isnan(y[3, 500].float()) and not y[3, :500].float().any()   # 1 / inf


@pytest.mark.parametrize("M,d", [(1, 8), (5, 264), (96, 5120), (777, 2560), (3, 32768), (500, 128), (301, 384),
                                 (999, 1000)])
def test_quant(M, d):
    import block_draft_selection_b200 as bds
    rng = np.random.default_rng(M * d)
    X = rng.standard_normal((M, d)).astype(np.float32)
    X[0, :8] = 127 * np.array([1, 0.5, -0.5, 1.5, 2.5, -2.5, 126.5, 63.5]) / 127   # halves of every parity
    x = bits(X)
    vals = syn.bf16_bits_to_f32(x)
    for m in range(M):   # half the maximum: 63.5 steps
        a = np.abs(vals[m]).max()
        x[m, -1] = bits(np.float32([a / 2 if m & 1 else -a / 2]))[0]
    q, scale = bds.dflash_quant_i8(dev_bf16(x))
    qr, sr = oracle.quant_i8(x)
    np.testing.assert_array_equal(q.cpu().numpy(), qr)
    np.testing.assert_array_equal(scale.cpu().numpy(), sr.astype(np.float32))   # one division, rounded once


def test_halves_of_every_maximum():
    """Rows whose maximum takes every bf16 mantissa, each with its own half,
    a third and neighbours: the quantiser's rounding is the exact one."""
    import block_draft_selection_b200 as bds
    a = (128 + np.arange(128)).astype(np.float32)              # every mantissa
    X = np.zeros((128, 264), np.float32)
    X[:, 0] = a
    X[:, 1] = a / 2
    X[:, 2] = -a / 2
    X[:, 8:] = np.arange(256)[None, :] * a[:, None] / 254.0
    x = bits(X)
    q, _ = bds.dflash_quant_i8(dev_bf16(x))
    np.testing.assert_array_equal(q.cpu().numpy(), oracle.quant_i8(x)[0])
    g = bits((1 + np.arange(264) / 128.0).astype(np.float32))  # products of 16 bits
    q, _, _ = bds.dflash_rmsnorm_i8(dev_bf16(x), dev_bf16(g))
    np.testing.assert_array_equal(q.cpu().numpy(), oracle.rmsnorm_i8(x, g)[0])


def test_in_place():
    """h over the residual, and y over x, as a program updates its stream in place."""
    import block_draft_selection_b200 as bds
    x, res, g = _inputs(33, 4096, 1, True)
    dx, dr, dg = dev_bf16(x), dev_bf16(res), dev_bf16(g)
    y, h = bds.dflash_rmsnorm(dx, dg, residual=dr)
    dx2, dr2 = dx.clone(), dr.clone()
    y2, h2 = bds.dflash_rmsnorm(dx2, dg, residual=dr2, y=dx2, h=dr2)
    assert y2 is dx2 and h2 is dr2 and torch.equal(y, y2) and torch.equal(h, h2)
    with pytest.raises(bds.DFlashError):
        bds.dflash_rmsnorm(dx, dg, residual=dr, y=dr, h=dr)


def test_rows_past_32_bit_offsets():
    import block_draft_selection_b200 as bds
    M, d = 66000, 32768                                        # 2.16e9 elements
    x = torch.zeros((M, d), dtype=torch.bfloat16, device="cuda")
    rows = [0, 65535, 65999]
    src, _, _ = _inputs(3, d, 2, False)
    x[rows] = dev_bf16(src)
    q, scale = bds.dflash_quant_i8(x)
    np.testing.assert_array_equal(q[rows].cpu().numpy(), oracle.quant_i8(src)[0])
    assert not scale[1:65535].any()


def test_shapes_and_types_refused():
    import block_draft_selection_b200 as bds
    x, res, g = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((4, 64), (4, 64), (64,)))
    with pytest.raises(ValueError):
        bds.dflash_rmsnorm(x[:, :32], g[:32])                  # not contiguous
    with pytest.raises(ValueError):
        bds.dflash_rmsnorm(x, g[:32])
    with pytest.raises(ValueError):
        bds.dflash_rmsnorm(x, g, h=res)                        # no residual
    with pytest.raises(TypeError):
        bds.dflash_rmsnorm(x.float(), g)
    with pytest.raises(TypeError):
        bds.dflash_rmsnorm_i8(x, g, q=torch.zeros(4, 64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        bds.dflash_quant_i8(x[0])
    with pytest.raises(bds.DFlashError):
        bds.dflash_rmsnorm(x, g, eps=0.0)
    with pytest.raises(bds.DFlashError):
        bds.dflash_quant_i8(torch.zeros(4, 12, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(bds.DFlashError):
        bds.dflash_quant_i8(x[:0])
