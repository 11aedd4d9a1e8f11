"""The int8 matrix product on the GPU: every element must equal the oracle's,
bit for bit -- the integer sum is exact, and the roundings to fp32 (the sum's,
one per scale) and to bf16 are part of the definition."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


def _inputs(M, N, K, seed, full=False):
    rng = np.random.default_rng(seed)
    if full:
        A, B = rng.integers(-128, 128, (M, K)), rng.integers(-128, 128, (N, K))
    else:
        A = np.clip(np.rint(rng.standard_normal((M, K)) * 32), -127, 127)
        B = np.clip(np.rint(rng.standard_normal((N, K)) * 32), -127, 127)
    sa = (0.01 + 0.02 * rng.random(M)).astype(np.float32)
    sb = (0.01 + 0.02 * rng.random(N)).astype(np.float32)
    return A.astype(np.int8), sa, B.astype(np.int8), sb


def _dev(*arrays):
    return [torch.from_numpy(a).cuda() for a in arrays]


def _run(A, sa, B, sb, dtype=torch.float32, **kw):
    import block_draft_selection_b200 as bds
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    C = bds.dflash_gemm_i8(*_dev(A, sa, B, sb), dtype=dtype, dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    return C


# around every tile edge of 16, 32, 64, 128 and 256 rows, K from one step to many, odd and even outer sizes
SHAPES = [(1, 1, 16), (1, 17, 64), (8, 4096, 256), (7, 2560, 2560), (15, 1000, 144), (16, 129, 128), (17, 128, 112),
          (33, 4099, 272), (64, 300, 1040), (127, 257, 128), (128, 640, 400), (129, 255, 256), (130, 2049, 272),
          (160, 33, 96), (192, 16, 512), (255, 513, 128), (256, 256, 256), (257, 1000, 384), (300, 4099, 160),
          (448, 1030, 640), (512, 31, 2576), (1000, 777, 208), (2049, 129, 64), (3, 40000, 80), (100, 19000, 64),
          # few tiles, K over a cluster: two, four and eight CTAs to a tile, parts of unequal length
          (1, 64, 5120), (8, 70, 1040), (128, 16, 5120), (100, 2560, 2560), (16, 1000, 272), (128, 1027, 1936),
          (5, 2000, 400), (65, 4500, 1168),
          # more than 128 tokens in few tiles, and so many that pairs take them
          (130, 300, 2576), (192, 1024, 5120), (600, 600, 1040), (1000, 300, 2064), (145, 1003, 4112), (130, 38500, 80),
          (333, 20001, 144), (1500, 5003, 272), (2500, 2051, 400),
          # few channels: rows of A as the long operand, alone and over a cluster
          (300, 1, 5120), (129, 100, 96), (200, 70, 2576), (1000, 5, 1552), (4352, 5, 1040), (2000, 128, 272),
          (5000, 17, 640), (40000, 3, 80), (50001, 128, 16)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    A, sa, B, sb = _inputs(M, N, K, M * 7 + N + K)
    ref = oracle.gemm_i8(A, sa, B, sb)
    np.testing.assert_array_equal(_run(A, sa, B, sb).cpu().numpy(), ref)
    want = torch.from_numpy(ref).bfloat16()
    assert torch.equal(_run(A, sa, B, sb, torch.bfloat16).cpu(), want)


@pytest.mark.parametrize("M,N,K", [(130, 300, 160), (256, 1000, 384), (300, 4099, 272), (1000, 777, 208)])
def test_product_without_pairs(M, N, K, monkeypatch):
    """DFLASH_PAIR=0 (read at every call): single CTAs on the tensor-bound path."""
    monkeypatch.setenv("DFLASH_PAIR", "0")
    A, sa, B, sb = _inputs(M, N, K, 5)
    np.testing.assert_array_equal(_run(A, sa, B, sb).cpu().numpy(), oracle.gemm_i8(A, sa, B, sb))


@pytest.mark.parametrize("M", [5, 200])
def test_largest_sums(M):
    """Every product 128 * 128, K at its limit: the int32 sum reaches 2^31 - 2^18."""
    K = 131056
    A = np.full((M, K), -128, np.int8)
    B = np.full((70, K), -128, np.int8)
    B[1::2, :] = 127
    one = np.ones
    C = _run(A, one(M, np.float32), B, one(70, np.float32)).cpu().numpy()
    assert (C[:, ::2] == np.float32(128 * 128 * K)).all() and (C[:, 1::2] == np.float32(-128 * 127 * K)).all()


@pytest.mark.parametrize("M,N,K", [(9, 3000, 512), (300, 500, 512)])
def test_full_range_values(M, N, K):
    A, sa, B, sb = _inputs(M, N, K, 1, full=True)
    np.testing.assert_array_equal(_run(A, sa, B, sb).cpu().numpy(), oracle.gemm_i8(A, sa, B, sb))


@pytest.mark.parametrize("M,N", [(6, 300), (260, 300), (300, 60), (30000, 60)])
def test_scales_as_they_are(M, N):
    """Zero, negative, infinite and NaN scales reach exactly their rows and columns."""
    A, sa, B, sb = _inputs(M, N, 128, 2)
    sa[:5] = [0.0, -1.5, np.inf, np.nan, 1e-30]
    sb[7], sb[N - 1] = np.nan, -2.0
    with np.errstate(invalid="ignore"):
        ref = oracle.gemm_i8(A, sa, B, sb)
    got = _run(A, sa, B, sb).cpu().numpy()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
    np.testing.assert_array_equal(got[~np.isnan(ref)], ref[~np.isnan(ref)])
    assert np.isnan(got[3]).all() and np.isnan(got[:, 7]).all()


@pytest.mark.parametrize("M,N", [(8, 1003), (200, 1003), (200, 1004), (1003, 101), (40001, 7)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_output_at_any_element(M, N, dtype):
    """C inside a larger buffer, aligned to its element only; nothing around it changes."""
    A, sa, B, sb = _inputs(M, N, 272, 4)
    buf = torch.full((M * N + 9,), 7.0, dtype=dtype, device="cuda")
    C = buf[5:5 + M * N].view(M, N)
    _run(A, sa, B, sb, C=C)
    assert torch.equal(C.float().cpu(), torch.from_numpy(oracle.gemm_i8(A, sa, B, sb)).to(dtype).float())
    assert (buf[:5] == 7).all() and (buf[5 + M * N:] == 7).all()


def test_repeatable():
    A, sa, B, sb = _inputs(130, 5000, 2576, 6)
    first = _run(A, sa, B, sb)
    for _ in range(3):
        assert torch.equal(_run(A, sa, B, sb), first)


@pytest.mark.parametrize("M,N", [(17000, 129280), (100, 21600000), (21600000, 100)])
def test_output_past_32_bit_offsets(M, N):
    """More than 2^31 elements of C: the last rows and columns are checked."""
    import block_draft_selection_b200 as bds
    K = 16
    g = torch.Generator(device="cuda").manual_seed(1)
    A = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    B = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    C = bds.dflash_gemm_i8(A, sa, B, sb, dtype=torch.bfloat16)
    for rows, cols in ((slice(M - 40, M), slice(N - 500, N)), (slice(0, 40), slice(0, 500)),
                       (slice(M // 2, M // 2 + 40), slice(N // 2, N // 2 + 500))):
        ref = oracle.gemm_i8(A[rows].cpu().numpy(), sa[rows].cpu().numpy(), B[cols].cpu().numpy(), sb[cols].cpu().numpy())
        assert torch.equal(C[rows, cols].cpu(), torch.from_numpy(ref).bfloat16())


def test_shapes_and_types_refused():
    import block_draft_selection_b200 as bds
    A, sa, B, sb = _dev(*_inputs(4, 32, 64, 0))
    for bad, err in (((A.float(), sa, B, sb), TypeError), ((A, sa.double(), B, sb), TypeError),
                     ((A, sa[:3], B, sb), ValueError), ((A, sa, B[:, :32], sb), ValueError),
                     ((A, sa, B.t(), sb), ValueError), ((A.cpu(), sa, B, sb), TypeError)):
        with pytest.raises(err):
            bds.dflash_gemm_i8(*bad)
    with pytest.raises(TypeError):
        bds.dflash_gemm_i8(A, sa, B, sb, dtype=torch.float16)
    with pytest.raises(ValueError):
        bds.dflash_gemm_i8(A, sa, B, sb, C=torch.empty(4, 31, device="cuda"))
    with pytest.raises(bds.DFlashError):
        bds.dflash_gemm_i8(A[:, :24].contiguous(), sa, B[:, :24].contiguous(), sb)     # K % 16
    with pytest.raises(bds.DFlashError):
        bds.dflash_gemm_i8(A[:0], sa[:0], B, sb)


def test_calls_at_once_and_replayed():
    """Products of every form on three streams at once, and captured and replayed with new inputs."""
    import block_draft_selection_b200 as bds
    cases = [_inputs(M, N, K, M + N) for M, N, K in ((8, 64, 5120), (600, 600, 1040), (4352, 5, 1040), (96, 20000, 256),
                                                     (448, 5000, 640))]
    refs = [torch.from_numpy(oracle.gemm_i8(*c)) for c in cases]
    dev = [_dev(*c) for c in cases]
    outs = [[torch.empty(c[0].shape[0], c[2].shape[0], device="cuda") for c in cases] for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, stream in enumerate(streams):
            for i in range(len(cases)):
                bds.dflash_gemm_i8(*dev[(i + s) % len(cases)], C=outs[s][(i + s) % len(cases)], stream=stream)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(c.cpu(), r) for c, r in zip(o, refs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [bds.dflash_gemm_i8(*d) for d in dev]
    for d in dev:
        d[0].neg_()                                            # values in [-127, 127]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(c.cpu(), -r) for c, r in zip(captured, refs))
