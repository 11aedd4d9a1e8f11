"""Pins of the oracle's norm, int8 and log-probability functions (CPU)."""
import math
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest

import oracle
import block_draft_synth as syn

bits = syn.f32_to_bf16_bits
vals = syn.bf16_bits_to_f32


def test_rmsnorm_hand_row():
    # h = (3, -4, 0, ...): sum of squares 25 over 16 channels; eps 0 leaves r = 4/5
    x = np.zeros((1, 16), np.float32)
    x[0, :2] = [3, -4]
    g = np.ones(16, np.float32)
    g[1] = 2.0
    y, h, r = oracle.rmsnorm(bits(x), bits(g), eps=0.0)
    assert r[0] == pytest.approx(0.8, rel=1e-15)
    np.testing.assert_allclose(y[0, :3], [2.4, -6.4, 0.0], rtol=1e-15)
    q, scale, _ = oracle.rmsnorm_i8(bits(x), bits(g), eps=0.0)
    assert q[0, :3].tolist() == [48, -127, 0]           # 127 * 3 / 8 = 47.625
    assert scale[0] == pytest.approx(6.4 / 127, rel=1e-15)


def test_residual_sum_rounds_once_to_bf16():
    # 1 + 2^-8 lies halfway between two bf16 values: ties to even (1); 1 + 3 * 2^-8 to 1 + 2^-6
    x = bits(np.array([[1.0, 1.0, 256.0]], np.float32))
    res = bits(np.array([[2.0 ** -8, 3 * 2.0 ** -8, 1.0]], np.float32))
    assert oracle.residual_sum(x, res)[0].tolist() == [1.0, 1.0 + 2.0 ** -6, 256.0]


def test_quantiser_rounds_every_quotient_exactly():
    """Against rational arithmetic, with rows made of halves: 127 times a
    power of two (every odd multiple of half a step is a tie) and half the
    maximum (the tie at 63.5 of any row)."""
    rng = np.random.default_rng(3)
    rows = [np.concatenate([[127.0], np.arange(31) + 0.5, -np.arange(32) - 0.5]) * s for s in (1.0, 2.0 ** -9)]
    for _ in range(6):
        r = vals(bits(rng.standard_normal(64).astype(np.float32)))
        r[7] = abs(r).max() / 2
        rows.append(r)
    X = np.stack([np.resize(np.asarray(r, np.float32), 64) for r in rows])
    Xb = bits(X)
    q, scale = oracle.quant_i8(Xb)
    for m, row in enumerate(vals(Xb)):
        a = max(abs(Fraction(float(v))) for v in row)
        for c, v in enumerate(row):
            t = 127 * Fraction(float(v)) / a
            lo = math.floor(t)
            want = lo if t - lo < Fraction(1, 2) else lo + 1 if t - lo > Fraction(1, 2) else lo + (lo & 1)
            assert q[m, c] == want, (m, c)
        assert scale[m] == float(a) / 127


def test_quantiser_zero_rows():
    q, scale = oracle.quant_i8(bits(np.array([[0.0] * 8, [2.0 ** -101] * 8], np.float32)))
    assert not q.any() and not scale.any()


def test_gemm_exact_integers():
    rng = np.random.default_rng(0)
    A = rng.integers(-128, 128, (3, 48)).astype(np.int8)
    B = rng.integers(-128, 128, (5, 48)).astype(np.int8)
    A[0], B[0] = -128, -128
    sa, sb = np.ones(3, np.float32), np.ones(5, np.float32)
    c = oracle.gemm_i8(A, sa, B, sb)
    for m in range(3):
        for n in range(5):
            assert int(c[m, n]) == sum(int(a) * int(b) for a, b in zip(A[m], B[n]))
    assert c[0, 0] == 48 * 128 * 128
    s = oracle.gemm_i8(A, np.full(3, 0.5, np.float32), B, np.arange(5, dtype=np.float32))
    np.testing.assert_array_equal(s, c * 0.5 * np.arange(5))


def test_logprobs_against_decimal():
    getcontext().prec = 50
    z = np.array([[0.5, -1.25, 3.0, 3.0, -7.0]])
    for T in (0.5, 1.0, 2.0):
        e = [(Decimal(float(v)) / Decimal(T)).exp() for v in z[0]]
        p = [x / sum(e) for x in e]
        o = oracle.token_logprobs(z, [1], T, K=3)
        assert o["logp"][0] == pytest.approx(float(p[1].ln()), rel=1e-14)
        assert o["entropy"][0] == pytest.approx(float(-sum(x * x.ln() for x in p)), rel=1e-13)
        assert o["lse"][0] == pytest.approx(float(sum(e).ln()), rel=1e-14)
        assert o["rank"][0] == 4
        assert o["top_idx"][0].tolist() == [2, 3, 0]      # equal values: the lower index first
        np.testing.assert_allclose(o["top_logp"][0], [float(p[i].ln()) for i in (2, 3, 0)], rtol=1e-14)


def test_logprobs_closed_forms():
    V = 1000
    o = oracle.token_logprobs(np.zeros((1, V)), [7], 1.0, K=4)
    assert o["logp"][0] == pytest.approx(-math.log(V)) and o["entropy"][0] == pytest.approx(math.log(V))
    assert o["rank"][0] == 1 and o["top_idx"][0].tolist() == [0, 1, 2, 3]
    o = oracle.token_logprobs(np.full((1, V), np.finfo(np.float32).min), [7], 1.0, K=1)   # a mask's lowest value
    assert o["logp"][0] == pytest.approx(-math.log(V)) and o["entropy"][0] == pytest.approx(math.log(V))
    one = np.full((1, V), -np.inf)
    o = oracle.token_logprobs(one, [7], 1.0, K=2)          # nothing left by the mask
    assert o["logp"][0] == -np.inf and o["lse"][0] == -np.inf and o["entropy"][0] == 0
    one[0, 9] = -3.0
    o = oracle.token_logprobs(one, [9], 1.0, K=2)          # one token left
    assert o["logp"][0] == 0 and o["entropy"][0] == 0 and o["lse"][0] == -3.0
    assert o["top_idx"][0].tolist() == [9, 0] and o["top_logp"][0].tolist() == [0.0, -np.inf]


def test_emitted_tokens_and_a_planted_shift():
    draft = np.array([[10, 11, 12], [20, 21, 22]])
    accept, nxt = np.array([1, 3]), np.array([19, 29])
    t = oracle.emitted_tokens(draft, accept, nxt)
    assert t.tolist() == [19, -1, -1, -1, 20, 21, 29, -1]
    full = oracle.emitted_tokens(draft, np.array([4, 4]), nxt)
    assert full.tolist() == [10, 11, 12, 19, 20, 21, 22, 29]
    # a reading that scores token i against row i + 1 would differ
    z = np.random.default_rng(1).standard_normal((8, 40))
    a = oracle.token_logprobs(z, t, 1.0, 1)["logp"]
    b = oracle.token_logprobs(z, np.roll(t, 1), 1.0, 1)["logp"]
    assert np.abs(a - b).max() > 0.1
