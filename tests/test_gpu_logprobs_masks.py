"""Log-probabilities where logits are large in magnitude: masks by a finite
constant of any size, and rows that lie far from zero as a whole.

Every launch form is met: `copies` repeats the rows until their number asks
for it (clusters of CTAs of 512 threads, one or two CTAs of 256, 128 and 64
threads).  The bounds are those of test_gpu_logprobs with 8 more in |t|: the
reference is a product rounded to fp32 below 2^28, so that a row's largest
value may lie 8 from it."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

MASKS = [-1e4, -1e5, -1e9, -1e10, -1e12, -1e20, -1e28, -1e30, -3e38]
# (V, copies of the 14 rows), fp32 and bf16 fall into the same form but for the length of a vector
FORMS = [(3, 1), (40, 1), (1000, 1), (5003, 1), (140000, 1), (9000, 12), (20000, 20), (40000, 20), (5000, 25), (20000, 70), (900, 25),
         (3000, 90)]


def _tol(V):
    t = math.log2(V) + 72
    s = (4 + 2 * t * math.log(2) + V / 256 + 8) * 2.0 ** -24
    return s, 2 * s * (1 + t)


def _close(got, want, tol):
    got = got.double().cpu().numpy()
    want = np.where(np.abs(want) > np.finfo(np.float32).max, np.copysign(np.inf, want), want)
    fine = np.isfinite(want)
    np.testing.assert_array_equal(got[~fine], want[~fine])
    bad = ~(np.abs(got[fine] - want[fine]) <= tol + 2.0 ** -24 * np.abs(want[fine]))
    assert not bad.any(), (got[fine][bad][:5], want[fine][bad][:5], tol)


def _compare(out, ref, V, copies):
    logp, rank, ent, lse, tl, ti = (t.cpu() for t in out)
    s, e = _tol(V)
    for got, name, tol in ((logp, "logp", s), (lse, "lse", s), (ent, "entropy", e), (tl, "top_logp", s)):
        _close(got, np.concatenate([ref[name]] * copies), tol)
    np.testing.assert_array_equal(rank.numpy(), np.concatenate([ref["rank"]] * copies))
    np.testing.assert_array_equal(ti.numpy(), np.concatenate([ref["top_idx"]] * copies))


def _rows(V, mask, dtype, seed):
    """14 rows: the mask over an end, the other end, the middle, half and most
    of the vocabulary at random, all but one token, everything; rows of the
    constant with one or a few values near it; its negative; whole rows moved
    out to it."""
    rng = np.random.default_rng(seed)
    z = (2.5 * rng.standard_normal((14, V))).astype(np.float32)
    z[0, V // 2:] = mask
    z[1, :V - V // 8 - 1] = mask
    z[2, V // 8:V - V // 8] = mask
    z[3, rng.random(V) < 0.5] = mask
    z[4, rng.random(V) < 0.97] = mask
    z[5, np.arange(V) != V // 2] = mask
    z[6] = mask
    z[7] = mask
    z[7, V // 3] = np.nextafter(np.float32(mask), np.float32(0)) if dtype is torch.float32 else mask * 0.99
    z[8] = 2 * np.float32(mask) if mask > -1e38 else mask
    z[8, V // 3:V // 2 + 1] = mask
    z[9, V // 2] = -mask
    z[10] = -np.float32(mask)
    z[11] += np.float32(mask)
    z[12] -= np.float32(mask)
    z[13, ::2] = mask
    z[13, 1::2] = -math.inf
    return torch.from_numpy(z).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,copies", FORMS)
def test_finite_masks(V, copies, dtype):
    import block_draft_selection_b200 as bds
    for n, mask in enumerate(MASKS):
        T = (0.3, 0.5, 0.7, 1.0, 1.7)[(n + V + copies) % 5]
        z = _rows(V, mask, dtype, V + n)
        tok = np.full(14, V // 2, np.int32)
        K = min(16, V)
        out = bds.dflash_token_logprobs(z.cuda().repeat(copies, 1), torch.from_numpy(tok).cuda().repeat(copies), K=K,
                                        temperature=T)
        _compare(out, oracle.token_logprobs(z.double().numpy(), tok, float(np.float32(T)), K), V, copies)


@pytest.mark.parametrize("T", [0.3, 0.5, 0.7, 1.0])
@pytest.mark.parametrize("mask", MASKS)
def test_masks_and_temperatures(mask, T):
    """Each constant at each temperature (which products are rounded up and which down changes with both)."""
    import block_draft_selection_b200 as bds
    V = 20000
    z = _rows(V, mask, torch.float32, 5)
    tok = np.full(14, V // 3, np.int32)
    out = bds.dflash_token_logprobs(z.cuda(), torch.from_numpy(tok).cuda(), K=16, temperature=T)
    _compare(out, oracle.token_logprobs(z.double().numpy(), tok, float(np.float32(T)), 16), V, 1)


@pytest.mark.parametrize("T", [1e-6, 1e-5, 1e-3])
def test_small_temperatures(T):
    """z / T up to 1e9 with ordinary logits: the largest token alone, or all of a tie."""
    import block_draft_selection_b200 as bds
    V = 5000
    z = (10 * np.random.default_rng(2).standard_normal((8, V))).astype(np.float32)
    z[1, 7], z[2, 4000], z[2, 17] = 900.0, 60.0, 60.0
    z[3, ::50] = 150.0
    z[4, ::50] = 50.0
    z[5] -= 2000.0
    tok = z.argmax(axis=1).astype(np.int32)
    out = bds.dflash_token_logprobs(torch.from_numpy(z).cuda(), torch.from_numpy(tok).cuda(), K=16, temperature=T)
    _compare(out, oracle.token_logprobs(z.astype(np.float64), tok, float(np.float32(T)), 16), V, 1)


def test_emitted_rows_under_a_finite_mask():
    import block_draft_selection_b200 as bds
    B, L, V = 6, 4, 30000
    rng = np.random.default_rng(8)
    z = (2.5 * rng.standard_normal((B * (L + 1), V))).astype(np.float32)
    z[:, V // 4:] = -1e10
    draft = rng.integers(0, V // 4, (B, L)).astype(np.int32)
    nxt = rng.integers(0, V // 4, B).astype(np.int32)
    acc = rng.integers(1, L + 2, B).astype(np.int32)
    for dtype in (torch.float32, torch.bfloat16):
        t = torch.from_numpy(z).to(dtype)
        out = bds.dflash_emitted_logprobs(t.cuda(), *(torch.from_numpy(a).cuda() for a in (draft, acc, nxt)), K=16)
        ref = oracle.token_logprobs(t.double().numpy(), oracle.emitted_tokens(draft, acc, nxt), 1.0, 16)
        _compare([o.reshape(B * (L + 1), *o.shape[2:]) for o in out], ref, V, 1)
