"""Log-probabilities of given and of emitted tokens on the GPU against the
fp64 oracle.

Ranks and alternatives' indices must be equal (order by value, then index).
lse and log-probabilities: a term exp((z - ref) / T) carries 4 * 2^-24 of
exp2's error and 2 * 2^-24 |t| ln 2 of its exponent's (the difference's and
the product's roundings; |t| averages at most log2 V + 64 over the terms'
weight, the reference lagging by 64 at most), the sum at most one rounding of
2^-24 per term of a thread, V / 512 + 8 of them; an absolute error of log s,
to which the result's own rounding of 2^-24 comes.  The entropy is lse minus
the mean of t, whose relative error is that of its terms and of the sums once
more: twice as much, times 1 + |t|.  Temperature 1 / T is a product in fp64."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


def _tol(V):
    t = math.log2(V) + 64
    s = (4 + 2 * t * math.log(2) + V / 512 + 8) * 2.0 ** -24
    return s, 2 * s * (1 + t)


def _close(got, want, tol):
    """|got - want| <= tol + 2^-24 |want|; infinities and NaN equal.  A value
    beyond fp32's range (the difference of the type's lowest and largest
    value is twice its range) is an infinity in fp32."""
    got = got.double().cpu().numpy()
    want = np.where(np.abs(want) > np.finfo(np.float32).max, np.copysign(np.inf, want), want)
    fine = np.isfinite(want)
    np.testing.assert_array_equal(got[~fine], want[~fine])
    bad = np.abs(got[fine] - want[fine]) > tol + 2.0 ** -24 * np.abs(want[fine])
    assert not bad.any(), (got[fine][bad][:5], want[fine][bad][:5], tol)


def _compare(out, ref, V, shape=None):
    logp, rank, ent, lse, tl, ti = out
    flat = lambda t: t.reshape(-1, *t.shape[2:]) if shape else t
    s, e = _tol(V)
    _close(flat(logp), ref["logp"], s)
    _close(flat(lse), ref["lse"], s)
    _close(flat(ent), ref["entropy"], e)
    _close(flat(tl), ref["top_logp"], s)
    np.testing.assert_array_equal(flat(rank).cpu().numpy(), ref["rank"])
    np.testing.assert_array_equal(flat(ti).cpu().numpy(), ref["top_idx"])


def _call(z, tokens, K=16, T=1.0, **kw):
    import block_draft_selection_b200 as bds
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = bds.dflash_token_logprobs(z, tokens, K=K, temperature=T, dev_status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status)


def _logits(M, V, seed, dtype=torch.float32, pad=0):
    rng = np.random.default_rng(seed)
    z = (2.5 * rng.standard_normal((M, V + pad))).astype(np.float32)
    z[:, :3] += 8 * rng.random((M, min(3, V + pad)))
    t = torch.from_numpy(z).to(dtype).cuda()[:, :V]
    return t, t.double().cpu().numpy()


def _tokens(M, V, seed):
    t = np.random.default_rng(seed + 1).integers(0, V, M).astype(np.int32)
    return t, torch.from_numpy(t).cuda()


SIZES = [(1, 1, 0), (3, 2, 0), (2, 31, 1), (5, 33, 0), (4, 127, 2), (2, 512, 0), (3, 513, 3), (2, 4096, 0),
         (7, 4097, 0), (3, 8192, 5), (2, 8193, 0), (300, 1000, 24), (1, 151936, 0), (8, 151936, 0), (3, 151643, 293),
         (150, 32000, 0), (40, 70001, 0), (1, 1048576 + 3, 0)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V,pad", SIZES)
def test_rows(M, V, pad, dtype):
    z, z64 = _logits(M, V, M + V, dtype, pad)
    tok, dtok = _tokens(M, V, V)
    K = min(16, V)
    T = (1.0, 0.5, 2.0)[(M + V) % 3]
    out, status = _call(z, dtok, K, T)
    assert status == 0
    _compare(out, oracle.token_logprobs(z64, tok, T, K), V)


@pytest.mark.parametrize("T", [0.05, 0.7, 30.0])
@pytest.mark.parametrize("K", [0, 1, 5, 20, 32])
def test_alternatives_and_temperatures(K, T):
    M, V = 6, 20000
    z, z64 = _logits(M, V, K, torch.float32)
    tok, dtok = _tokens(M, V, 3)
    out, _ = _call(z, dtok, K, T)
    _compare(out, oracle.token_logprobs(z64, tok, T, K), V)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,copies", [(40, 1), (5000, 1), (140000, 1), (40, 90), (1000, 1), (1000, 20), (1500, 90),
                                      (4000, 30), (4000, 90), (9000, 80), (20000, 60)])
def test_masks_and_orders(V, copies, dtype):
    """Rows a mask leaves nothing, one or two tokens of; the lowest and the
    largest value of the type; constant rows; ties; rising and falling rows;
    +0 and -0; a row with one certain token; the same many times over, in the
    forms for many rows.  (Threads of the smallest form sum V / 256 terms, not
    V / 512: the tolerance of a row twice as long.)"""
    lowest = torch.finfo(dtype).min
    rng = np.random.default_rng(V)
    M = 16
    z = torch.from_numpy((2 * rng.standard_normal((M, V))).astype(np.float32)).to(dtype)
    z[0] = -math.inf
    z[1] = -math.inf
    z[1, V - 1] = -4.0
    z[2] = -math.inf
    z[2, V // 2] = z[2, V // 3] = 1.0
    z[3] = lowest
    z[4] = 0.25
    z[5] = lowest
    z[5, V // 2] = 3.0
    z[6, torch.from_numpy(rng.random(V) < 0.5)] = -math.inf
    z[7, torch.from_numpy(rng.random(V) < 0.5)] = lowest
    z[8] = torch.linspace(-20, 20, V).to(dtype)
    z[9] = torch.linspace(20, -20, V).to(dtype)
    z[10] = torch.from_numpy(rng.integers(-3, 4, V).astype(np.float32)).to(dtype)
    z[11] = 0.0
    z[11, ::2] = -0.0
    z[12, V // 2] = 90.0
    z[13] = torch.finfo(dtype).max
    z[14] = lowest
    z[14, 5] = torch.finfo(dtype).max
    z[15] = -60.0
    tok = np.full(M, V // 2, np.int32)
    K = 32
    ref = oracle.token_logprobs(z.double().numpy(), tok, 1.0, K)
    out, status = _call(z.cuda().repeat(copies, 1), torch.from_numpy(tok).cuda().repeat(copies), K)
    assert status == 0
    _compare(out, {k: np.concatenate([v] * copies) for k, v in ref.items()}, 2 * V if copies > 1 else V)
    assert out[0][0] == -math.inf and out[3][0] == -math.inf and out[2][0] == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nan_and_infinity(dtype):
    """A NaN or +inf reaches its own row's log-probabilities alone; a NaN leads the alternatives."""
    M, V, K = 6, 3001, 4
    z, z64 = _logits(M, V, 8, dtype)
    tok, dtok = _tokens(M, V, 8)
    z[1, 2500] = math.nan
    z[3, 17] = math.inf
    z[5] = math.nan
    out, _ = _call(z, dtok, K)
    logp, rank, ent, lse, tl, ti = [t.cpu() for t in out]
    for m in (1, 3, 5):
        assert torch.isnan(logp[m]) and torch.isnan(ent[m]) and torch.isnan(lse[m]) and torch.isnan(tl[m]).all()
    ok = [0, 2, 4]
    ref = oracle.token_logprobs(z64[ok], tok[ok], 1.0, K)
    _compare([t[ok] for t in out], ref, V)
    assert ti[1, 0] == 2500 and ti[3, 0] == 17 and ti[5].tolist() == [0, 1, 2, 3]
    order = np.lexsort((np.arange(V), -z64[1]))
    assert ti[1, 1:].tolist() == [v for v in order if v != 2500][:3]


@pytest.mark.parametrize("M,V", [(9, 5000), (9, 500), (300, 900), (1900, 300)])
def test_rows_not_asked_for_keep_what_they_held(M, V):
    K = 16
    z, z64 = _logits(M, V, 1)
    tok, _ = _tokens(M, V, 1)
    tok[[0, 4, 8]] = [-1, -100, -1]
    z[4] = math.nan
    outs = dict(logp=torch.full((M,), 7.0), rank=torch.full((M,), 7, dtype=torch.int32), entropy=torch.full((M,), 7.0),
                lse=torch.full((M,), 7.0), top_logp=torch.full((M, K), 7.0),
                top_idx=torch.full((M, K), 7, dtype=torch.int32))
    outs = {k: v.cuda() for k, v in outs.items()}
    out, status = _call(z, torch.from_numpy(tok).cuda(), K, **outs)
    assert status == 0
    for given, t in zip(outs.values(), out):
        assert t is given and (t[[0, 4, 8]] == 7).all()
    keep = tok >= 0
    ref = oracle.token_logprobs(z64[keep], tok[keep], 1.0, K)
    _compare([t[torch.from_numpy(keep).cuda()] for t in out], ref, V)
    fresh, _ = _call(z, torch.from_numpy(tok).cuda(), K)
    assert not fresh[0][0] and not fresh[5][8].any()          # what the call allocates is zero there


def test_padding_among_rows_that_clusters_share():
    """Few long rows, several CTAs to each: rows not asked for leave their outputs alone."""
    M, V, K = 6, 151936, 20
    z, z64 = _logits(M, V, 21)
    tok, _ = _tokens(M, V, 21)
    tok[[0, 3, 5]] = -1
    top = torch.full((M, K), 7, dtype=torch.int32, device="cuda")
    for _ in range(3):
        out, status = _call(z, torch.from_numpy(tok).cuda(), K, top_idx=top)
        assert status == 0 and (top[[0, 3, 5]] == 7).all()
        keep = tok >= 0
        ref = oracle.token_logprobs(z64[keep], tok[keep], 1.0, K)
        _compare([t[torch.from_numpy(keep).cuda()] for t in out], ref, V)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V", [(200, 9000), (500, 12345), (3, 100000), (20, 2000), (330, 1000), (1300, 3000),
                                 (1000, 40000)])
def test_rows_that_defeat_the_filter(M, V, dtype):
    """Rising rows and rows of one value, in every launch form: each value
    passes the bound that was known when it came."""
    z = torch.linspace(-30, 30, V).repeat(M, 1)
    z[1::3] = torch.arange(V) * 2.0 ** -10
    z[2::3] = 1.5
    z = z.to(dtype)
    tok = np.arange(M, dtype=np.int32)
    out, _ = _call(z.cuda(), torch.from_numpy(tok).cuda(), 20, 0.7)
    rows = [0, 1, 2, M - 1]
    ref = oracle.token_logprobs(z[rows].double().numpy(), tok[rows], 0.7, 20)
    _compare([t[rows] for t in out], ref, V)


def test_longest_row():
    V = 1 << 24
    g = torch.Generator().manual_seed(0)
    z = torch.randn((1, V), generator=g) * 2
    out, _ = _call(z.cuda(), torch.tensor([V - 1], dtype=torch.int32).cuda(), 8)
    z64 = z.double().numpy()
    lp, lse, ent = oracle.row_logprobs(z64[0])
    s, e = _tol(V)
    _close(out[0], lp[-1:], s)
    _close(out[2], np.array([ent]), e)
    _close(out[3], np.array([lse]), s)
    best = np.argpartition(-z64[0], 20)[:20]
    order = sorted(best, key=lambda v: (-z64[0, v], v))[:8]
    assert out[5][0].tolist() == order
    assert int(out[1]) == 1 + int((z64[0] > z64[0, -1]).sum())


def test_token_outside_the_vocabulary():
    import block_draft_selection_b200 as bds
    M, V = 4, 700
    z, z64 = _logits(M, V, 2, pad=30)
    tok = np.array([5, V, 6, 2 ** 31 - 1], np.int32)
    out, status = _call(z, torch.from_numpy(tok).cuda(), 8)
    assert status == bds.DFLASH_ERR_BAD_INDEX
    assert torch.isnan(out[0][[1, 3]]).all() and out[1][[1, 3]].tolist() == [0, 0]
    tok[[1, 3]] = 0
    ref = oracle.token_logprobs(z64, tok, 1.0, 8)
    ref["logp"][[1, 3]], ref["rank"][[1, 3]] = np.nan, 0
    _compare(out, ref, V)


def test_without_tokens():
    M, V = 5, 9000
    z, z64 = _logits(M, V, 4)
    out, _ = _call(z, None, 16)
    ref = oracle.token_logprobs(z64, np.zeros(M, int), 1.0, 16)
    assert out[0] is None and out[1] is None
    s, e = _tol(V)
    _close(out[2], ref["entropy"], e)
    _close(out[3], ref["lse"], s)
    np.testing.assert_array_equal(out[5].cpu().numpy(), ref["top_idx"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,L,V,pad", [(1, 1, 64, 0), (1, 7, 151936, 0), (16, 5, 5000, 3), (40, 16, 3000, 0),
                                       (3, 32, 4097, 0), (90, 16, 700, 1)])
def test_emitted(B, L, V, pad, dtype):
    import block_draft_selection_b200 as bds
    z, z64 = _logits(B * (L + 1), V, B + L, dtype, pad)
    rng = np.random.default_rng(L)
    draft = rng.integers(0, V, (B, L)).astype(np.int32)
    nxt = rng.integers(0, V, B).astype(np.int32)
    acc = rng.integers(1, L + 2, B).astype(np.int32)
    acc[:2] = [1, L + 1][:len(acc[:2])]
    d = [torch.from_numpy(a).cuda() for a in (draft, acc, nxt)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = bds.dflash_emitted_logprobs(z, *d, K=16, temperature=0.8, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert out[0].shape == (B, L + 1) and out[5].shape == (B, L + 1, 16)
    ref = oracle.token_logprobs(z64, oracle.emitted_tokens(draft, acc, nxt), 0.8, 16)
    _compare(out, ref, V, shape=True)


def test_emitted_out_of_range():
    import block_draft_selection_b200 as bds
    B, L, V = 3, 2, 100
    z, z64 = _logits(B * (L + 1), V, 1)
    draft = np.array([[1, 2], [-5, 4], [5, 6]], np.int32)
    acc, nxt = np.array([9, 2, 0], np.int32), np.array([7, 8, 100], np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = bds.dflash_emitted_logprobs(z, *[torch.from_numpy(a).cuda() for a in (draft, acc, nxt)], K=3,
                                      dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == bds.DFLASH_ERR_BAD_INDEX
    # accepted lengths read as 3, 2 and 1; the tokens -5 and 100 have no probability
    t = np.array([1, 2, 7, 0, 8, -1, 0, -1, -1])
    ref = oracle.token_logprobs(z64, t, 1.0, 3)
    for m in (3, 6):
        ref["logp"][m], ref["rank"][m] = np.nan, 0
    _compare(out, ref, V, shape=True)


def test_rows_past_32_bit_offsets():
    M, V = 16500, 131072                                       # 2.16e9 elements
    z = torch.empty((M, V), dtype=torch.bfloat16, device="cuda")
    rows = [0, 16383, 16384, 16499]
    tok = np.full(M, -1, np.int32)
    tok[rows] = [5, 6, 7, 8]
    src, z64 = _logits(4, V, 3, torch.bfloat16)
    z[rows] = src
    out, _ = _call(z, torch.from_numpy(tok).cuda(), 16)
    ref = oracle.token_logprobs(z64, tok[rows], 1.0, 16)
    _compare([t[rows] for t in out], ref, V)


@pytest.mark.parametrize("M,V", [(5, 151936), (400, 800), (400, 8000)])
def test_repeatable(M, V):
    z, _ = _logits(M, V, 11, torch.bfloat16)
    _, tok = _tokens(M, V, 11)
    first, _ = _call(z, tok, 32, 0.7)
    for _ in range(5):
        for a, b in zip(first, _call(z, tok, 32, 0.7)[0]):
            assert torch.equal(a, b)


def test_arguments_refused():
    import block_draft_selection_b200 as bds
    z = torch.zeros(4, 100, device="cuda")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    for call, err in ((lambda: bds.dflash_token_logprobs(z.half(), t), TypeError),
                      (lambda: bds.dflash_token_logprobs(z.t(), t), ValueError),
                      (lambda: bds.dflash_token_logprobs(z[:1].expand(4, 100), t), ValueError),
                      (lambda: bds.dflash_token_logprobs(z[0], t), ValueError),
                      (lambda: bds.dflash_token_logprobs(z, t.long()), TypeError),
                      (lambda: bds.dflash_token_logprobs(z, t[:3]), ValueError),
                      (lambda: bds.dflash_token_logprobs(z, t, K=33), ValueError),
                      (lambda: bds.dflash_token_logprobs(z, t, K=-1), ValueError),
                      (lambda: bds.dflash_token_logprobs(z[:, :8], t, K=9), bds.DFlashError),
                      (lambda: bds.dflash_token_logprobs(z, t, temperature=0.0), bds.DFlashError),
                      (lambda: bds.dflash_token_logprobs(z, None, logp=z[:, 0].contiguous()), ValueError),
                      (lambda: bds.dflash_token_logprobs(z, t, lse=torch.zeros(3, device="cuda")), ValueError),
                      (lambda: bds.dflash_emitted_logprobs(z, t.view(2, 2), t[:2], t[:2]), ValueError),
                      (lambda: bds.dflash_token_logprobs(z[:0], t[:0]), bds.DFlashError)):
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("K", [0, 3])
def test_outputs_not_given(K):
    """Outputs the call allocates: their shapes and types, each contiguous and apart from the others, zero
    where no row asked; the same on a stream of the caller's."""
    import block_draft_selection_b200 as bds
    z, z64 = _logits(6, 77, 12)
    tok = np.array([3, -1, 0, 76, -1, 40], np.int32)
    dtok = torch.from_numpy(tok).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = torch.from_numpy(tok >= 0).cuda()
    ref = oracle.token_logprobs(z64[tok >= 0], tok[tok >= 0], 1.0, K)
    for stream in (None, side):
        out = bds.dflash_token_logprobs(z, dtok, K=K, stream=stream)
        torch.cuda.synchronize()
        types = [torch.float32, torch.int32, torch.float32, torch.float32, torch.float32, torch.int32]
        assert [t.dtype for t in out] == types and all(t.is_contiguous() for t in out)
        assert [tuple(t.shape) for t in out] == [(6,)] * 4 + [(6, K)] * 2
        assert all(not t[~keep].any() for t in out)
        _compare([t[keep] for t in out], ref, 77)
        kept = [t.clone() for t in out]
        for i, t in enumerate(out):
            t.fill_(9)
            assert all(torch.equal(out[j], kept[j]) for j in range(i + 1, 6))
