"""Pins of the oracle's norm and quantiser: unit rows and the sign's symmetry."""
import numpy as np
import pytest

import oracle
import block_draft_synth as syn

bits = syn.f32_to_bf16_bits


@pytest.mark.parametrize("d", [8, 264, 4096])
def test_unit_rows(d):
    """+-1 everywhere: the mean square is 1, so y = +-gamma / sqrt(1 + eps), q = +-127 and the scale 1 / 127."""
    sign = np.where(np.arange(d) % 3 == 0, -1.0, 1.0)
    x, one = bits(sign[None].astype(np.float32)), bits(np.ones(d, np.float32))
    y, h, r = oracle.rmsnorm(x, one, eps=0.0)
    assert r[0] == 1.0 and (y[0] == sign).all() and (h[0] == sign).all()
    y, _, _ = oracle.rmsnorm(x, one, eps=0.21)
    np.testing.assert_allclose(y[0], sign / 1.1, rtol=1e-15)
    q, scale, _ = oracle.rmsnorm_i8(x, one, eps=0.0)
    assert (q[0] == 127 * sign).all() and scale[0] == 1 / 127
    q, scale = oracle.quant_i8(x)
    assert (q[0] == 127 * sign).all() and scale[0] == 1 / 127


def test_sign_symmetry():
    """-x, or -gamma, gives -y and -q and the same scale."""
    rng = np.random.default_rng(7)
    v = rng.standard_normal((5, 264)).astype(np.float32)
    g = (1 + 0.3 * rng.standard_normal(264)).astype(np.float32)
    y, _, r = oracle.rmsnorm(bits(v), bits(g))
    q, s, _ = oracle.rmsnorm_i8(bits(v), bits(g))
    for a, b in ((-v, g), (v, -g)):
        y2, _, r2 = oracle.rmsnorm(bits(a), bits(b))
        q2, s2, _ = oracle.rmsnorm_i8(bits(a), bits(b))
        assert (y2 == -y).all() and (r2 == r).all() and (q2 == -q).all() and (s2 == s).all()
    k, t = oracle.quant_i8(bits(v))
    k2, t2 = oracle.quant_i8(bits(-v))
    assert (k2 == -k).all() and (t2 == t).all()
