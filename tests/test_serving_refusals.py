"""Refusals of the norm, int8 and log-probability entry points: on the host,
before any launch (no GPU; the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

INVALID = 1


@pytest.fixture(scope="module")
def lib():
    import block_draft_selection_b200 as bds
    return bds.lib


OK = 0x1000


def test_rmsnorm(lib):
    def call(x=OK, res=OK, g=OK, eps=1e-6, M=4, d=64, h=OK, y=OK + 0x1000):
        return lib.dflash_rmsnorm(x, res, g, eps, M, d, h, y, None)
    for bad in (dict(x=None), dict(g=None), dict(y=None), dict(M=0), dict(M=-1), dict(d=0), dict(d=12), dict(d=32776),
                dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-30),
                dict(x=OK + 8), dict(res=OK + 2), dict(g=OK + 4), dict(h=OK + 8), dict(y=OK + 8),
                dict(res=None), dict(h=OK + 0x1000)):
        assert call(**bad) == INVALID, bad


def test_rmsnorm_i8_and_quant(lib):
    def call(x=OK, res=OK, g=OK, eps=1e-6, M=4, d=64, h=OK, q=OK, s=OK):
        return lib.dflash_rmsnorm_i8(x, res, g, eps, M, d, h, q, s, None)
    for bad in (dict(x=None), dict(g=None), dict(q=None), dict(s=None), dict(M=0), dict(d=20), dict(eps=0.0),
                dict(q=OK + 4), dict(s=OK + 2), dict(res=None)):
        assert call(**bad) == INVALID, bad

    def quant(x=OK, M=4, d=64, q=OK, s=OK):
        return lib.dflash_quant_i8(x, M, d, q, s, None)
    for bad in (dict(x=None), dict(q=None), dict(s=None), dict(M=0), dict(d=20), dict(d=40000), dict(x=OK + 8),
                dict(q=OK + 4), dict(s=OK + 1)):
        assert quant(**bad) == INVALID, bad


def test_gemm_i8(lib):
    def call(A=OK, sa=OK, B=OK, sb=OK, C=OK, bf16=0, M=4, N=64, K=64):
        return lib.dflash_gemm_i8(A, sa, B, sb, C, bf16, M, N, K, None, None)
    for bad in (dict(A=None), dict(sa=None), dict(B=None), dict(sb=None), dict(C=None), dict(bf16=2), dict(M=0),
                dict(N=0), dict(K=0), dict(K=24), dict(K=131072), dict(A=OK + 8), dict(B=OK + 4), dict(sa=OK + 2),
                dict(sb=OK + 1), dict(C=OK + 2), dict(C=OK + 1, bf16=1)):
        assert call(**bad) == INVALID, bad


def test_token_logprobs(lib):
    def call(z=OK, bf16=0, ld=100, M=4, V=100, tok=OK, T=1.0, K=16, logp=OK, rank=OK, ent=OK, lse=OK, tl=OK, ti=OK):
        return lib.dflash_token_logprobs(z, bf16, ld, M, V, tok, T, K, logp, rank, ent, lse, tl, ti, None, None)
    for bad in (dict(z=None), dict(bf16=2), dict(ld=99), dict(M=0), dict(V=0), dict(V=(1 << 24) + 1, ld=1 << 25),
                dict(T=0.0), dict(T=-1.0), dict(T=float("inf")), dict(T=float("nan")), dict(T=1e-7), dict(T=2e6), dict(K=-1), dict(K=33),
                dict(K=16, V=10), dict(tok=None), dict(tok=None, logp=None), dict(tl=None), dict(ti=None), dict(K=0),
                dict(z=OK + 2), dict(z=OK + 1, bf16=1)):
        assert call(**bad) == INVALID, bad


def test_emitted_logprobs(lib):
    def call(z=OK, bf16=0, ld=100, B=4, L=3, V=100, draft=OK, acc=OK, nxt=OK, T=1.0, K=16, tl=OK, ti=OK):
        return lib.dflash_emitted_logprobs(z, bf16, ld, B, L, V, draft, acc, nxt, T, K, OK, OK, OK, OK, tl, ti, None,
                                           None)
    for bad in (dict(z=None), dict(draft=None), dict(acc=None), dict(nxt=None), dict(B=0), dict(L=0), dict(L=33),
                dict(B=1 << 30, L=31), dict(ld=99), dict(V=0), dict(T=0.0), dict(K=33), dict(ti=None)):
        assert call(**bad) == INVALID, bad


def test_binding_refuses_what_is_not_on_a_gpu():
    import block_draft_selection_b200 as bds
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    i8 = torch.zeros(4, 64, dtype=torch.int8)
    f = torch.zeros(4)
    for call in (lambda: bds.dflash_rmsnorm(x, x[0]), lambda: bds.dflash_rmsnorm_i8(x, x[0]),
                 lambda: bds.dflash_quant_i8(x), lambda: bds.dflash_gemm_i8(i8, f, i8, f),
                 lambda: bds.dflash_token_logprobs(f[None]),
                 lambda: bds.dflash_emitted_logprobs(f[None], i8, i8, i8)):
        with pytest.raises(TypeError):
            call()


def test_binding_matches_the_header():
    """ctypes signatures have as many arguments as the header declares."""
    import os
    import re
    import block_draft_selection_b200 as bds
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "dflash.h")).read(), flags=re.S)
    for name in ("dflash_rmsnorm", "dflash_rmsnorm_i8", "dflash_quant_i8", "dflash_gemm_i8", "dflash_token_logprobs",
                 "dflash_emitted_logprobs"):
        args = re.search(r"int " + name + r"\(([^)]*)\)", text).group(1).split(",")
        f = getattr(bds.lib, name)
        assert len(f.argtypes) == len(args), name
        for c, a in zip(f.argtypes, args):
            want = (ctypes.c_void_p if "*" in a else ctypes.c_float if "float" in a
                    else ctypes.c_longlong if "long long" in a else ctypes.c_int)
            assert c is want, (name, a)
