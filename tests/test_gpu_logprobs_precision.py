"""Precision and signs of log-probabilities and entropies, row by row.

The bounds follow the arithmetic for each row, from its own probabilities.
With t = (z - max) log2(e) / T <= 0, p the probabilities, p0 the largest
one, tbar = sum p |t| and t2 = sum p t^2:

- a term 2^t carries exp2's relative error, 4 * 2^-24, and that of its
  exponent's rounding, ln 2 |t| 2^-24;
- a sum of n terms in fp32 rounds n times by at most 2^-24 of itself, and
  each time by no more than the smaller addend (the larger one is
  representable), so by no more than 1 - p0 in all;
- when the reference moves by d (a record of the warp, once a round at most),
  the sums so far, which do not hold the record, take the error of 2^-d:
  (6 + ln 2 d) 2^-24, and d adds up to the rise of the row;
- log s: 2 * 2^-24 of its mantissa's part.

  error of log s   E = 2^-24 (6 + ln 2 tbar) + min(X 2^-24, 1 - p0)
  X = terms of an accumulator + 6 rounds + ln 2 rise + 13

to which the output's rounding comes.  The entropy is log s - ln 2 w / s with
w = sum p t: its terms carry their factors' errors, its sums the same X times
w, the quotient E once more, and the temperature's rounding 2^-24 t2 ln^2 2:

  error of entropy   E (1 + ln 2 tbar) + ln 2 2^-24 ((6 + 2 X) tbar + 2 ln 2 t2)

On random rows roundings are independent: for the X of them the root stands,
times 8 (more than eight deviations of a rounding's 2^-24 / sqrt 3 each)."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LN2 = math.log(2)


def _form(M, V, dtype, sms):
    """(threads, CTAs to a row) that the launch rule gives."""
    n_vec = (V * (4 if dtype is torch.float32 else 2) + 15) // 16
    if n_vec <= (1024 if M > 8 * sms else 256) and M > 2 * sms:
        return 64, 1
    if n_vec <= 512 or (n_vec <= 4096 and M > 2 * sms) or M > 6 * sms:
        return 128, 1
    if M <= sms:
        Q = 1
        while Q < 8 and 2 * Q * M <= sms and V // (2 * Q) >= 4096:
            Q *= 2
        return 512, Q
    return 256, 2 if 2 * M <= 3 * sms and V >= 8192 else 1


def _bounds(z, T, M, dtype, random):
    """(error of logp and lse, error of entropy) of each row of z [m, V]; M: rows of the call."""
    nt, Q = _form(M, z.shape[1], dtype, torch.cuda.get_device_properties(0).multi_processor_count)
    per_thread = z.shape[1] / (Q * nt)
    E, H = [], []
    for row in z:
        fine = row[np.isfinite(row)]
        t = (fine - fine.max()) / T / LN2
        e = np.exp2(t)
        p = e / e.sum()
        tail = (e.sum() - 1) / e.sum()
        tbar, t2 = (p * -t).sum(), (p * t * t).sum()
        rounds = math.ceil(per_thread / (16 if dtype is torch.float32 else 32)) + 1
        X = per_thread / 4 + 6 * rounds + LN2 * (-t.min()) + 13
        if random:
            X = 8 * math.sqrt(X)
        err = U * (6 + LN2 * tbar) + min(X * U, tail)
        E.append(err)
        H.append(err * (1 + LN2 * tbar) + LN2 * U * ((6 + 2 * X) * tbar + 2 * LN2 * t2))
    return np.array(E), np.array(H)


def _within(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert not np.isnan(got).any(), what
    if got.ndim == 2:
        tol = tol[:, None]
    err = np.abs(got - want) - U * np.abs(want)
    assert (err <= tol).all(), (what, (err / tol).max(), got[err > tol][:4], want[err > tol][:4])


def _check(z, tok, T, copies, random, K=16):
    import block_draft_selection_b200 as bds
    z64 = z.double().numpy()
    m, V = z.shape
    out = bds.dflash_token_logprobs(z.cuda().repeat(copies, 1), torch.from_numpy(tok).cuda().repeat(copies), K=K,
                                    temperature=T)
    T = float(np.float32(T))
    ref = oracle.token_logprobs(z64, tok, T, K)
    E, H = (np.concatenate([x] * copies) for x in _bounds(z64, T, m * copies, z.dtype, random))
    want = {k: np.concatenate([v] * copies) for k, v in ref.items()}
    logp, rank, ent, lse, tl, ti = (t.cpu() for t in out)
    _within(logp, want["logp"], E, "logp")
    _within(lse, want["lse"], E, "lse")
    _within(tl, want["top_logp"], E, "top_logp")
    _within(ent, want["entropy"], H, "entropy")
    assert (logp <= 0).all() and (tl <= 0).all() and (ent >= 0).all()
    np.testing.assert_array_equal(rank.numpy(), want["rank"])
    np.testing.assert_array_equal(ti.numpy(), want["top_idx"])


FORMS = [(1000, 1), (151936, 1), (9000, 20), (40000, 30), (5000, 40), (20000, 110), (900, 40), (3000, 150)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,copies", FORMS)
def test_one_token_above_the_others(V, copies, dtype):
    """8 rows, each with a token 10 to 60 above the body: in the first round,
    later, at the end; the token asked for is that one, but in the last row."""
    rng = np.random.default_rng(V)
    for T in (1.0, 0.7):
        z = (2.0 * rng.standard_normal((8, V))).astype(np.float32)
        at = [0, V // 2, V - 1, V // 3, 2 * V // 3, V - 5, V // 2 + 7, V // 4]
        z[np.arange(8), at] = [10, 20, 30, 35, 43, 60, 25, 32]
        z[7, V // 2:] = -np.inf
        tok = np.array(at, np.int32)
        tok[6] = 3
        _check(torch.from_numpy(z).to(dtype), tok, T, copies, False)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,copies", FORMS)
def test_random_rows(V, copies, dtype):
    """Ordinary rows, flat ones and steep ones, with a bound close to what independent roundings give."""
    rng = np.random.default_rng(V + 1)
    for T in (1.0, 0.6, 1.7):
        z = rng.standard_normal((8, V)) * np.array([0.1, 1, 2, 2.5, 3, 4, 6, 10])[:, None]
        z[:, :3] += 9 * rng.random((8, 3))
        _check(torch.from_numpy(z.astype(np.float32)).to(dtype), rng.integers(0, V, 8).astype(np.int32), T, copies,
               True)


@pytest.mark.parametrize("V,copies", [(5000, 1), (900, 60), (20000, 30)])
def test_rising_rows(V, copies):
    """Every round a record: the sums move to a new reference each time."""
    z = np.stack([np.linspace(-20, 20, V), np.linspace(-300, 300, V), np.linspace(0, 3000, V),
                  np.repeat(np.linspace(-40, 40, V // 50), 50)[:V]]).astype(np.float32)
    _check(torch.from_numpy(z), np.array([V - 1, V - 1, V - 1, 0], np.int32), 0.7, copies, False)


def test_certain_rows():
    """One token left by the mask, or one far above: log-probability 0 and entropy 0, never the other sign."""
    import block_draft_selection_b200 as bds
    V = 3000
    z = torch.full((4, V), -math.inf)
    z[0, 17] = 3.7
    z[1, V - 1] = -123.4
    z[2] = 0.3
    z[2, 2000] = 150.0
    z[3] = -1e9
    z[3, 5] = 11.3
    tok = torch.tensor([17, V - 1, 2000, 5], dtype=torch.int32)
    for T in (0.3, 0.7, 1.0, 1.9):
        logp, rank, ent, lse, tl, ti = bds.dflash_token_logprobs(z.cuda(), tok.cuda(), K=3, temperature=T)
        z32 = torch.tensor([3.7, -123.4, 150.0, 11.3])
        want = z32.double() / float(np.float32(T))
        assert ((lse.cpu().double() - want).abs() <= 6 * U + U * want.abs()).all()
        assert (logp.cpu() <= 0).all() and (logp.cpu() >= -6 * U).all()
        assert (ent.cpu() >= 0).all() and (ent.cpu() <= 6 * U).all()
        assert (tl[:, 0] == logp).all() and (rank == 1).all()
