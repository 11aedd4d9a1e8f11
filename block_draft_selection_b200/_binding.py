"""ctypes binding of libdflash.so: argument marshalling only.

Each function here has the name of the C entry point it calls, checks that
the torch tensors it is given are CUDA tensors of the layout the C ABI
documents (include/dflash.h), allocates outputs the caller did not pass, and
forwards raw device pointers and the current CUDA stream.  Every step of the
computation runs in the library's kernels; there is no CPU path.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdflash.so")

DFLASH_OK = 0
DFLASH_ERR_INVALID_ARG = 1
DFLASH_ERR_UNSUPPORTED = 2
DFLASH_ERR_CUDA = 3
DFLASH_ERR_WORKSPACE = 4
DFLASH_ERR_TIMEOUT = 5
DFLASH_ERR_BAD_INDEX = 6
K_TOP = 16


class DFlashError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {dflash_status_string(code)} (status {code})")
        self.code = code


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python block_draft_selection_b200/build.py` "
            "(this package has no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sig = {
        "dflash_status_string": (ctypes.c_char_p, [i32]),
        "dflash_build_id": (ctypes.c_char_p, []),
        "dflash_conv2tap": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, vp]),
        "dflash_lmhead_topk_workspace": (sz, [i32, i32, i32]),
        "dflash_lmhead_topk": (i32, [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp, vp]),
        "dflash_lmhead_logits_debug": (i32, [vp, vp, i32, i32, i32, vp, vp, sz, vp, vp]),
        "dflash_path_select": (i32, [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]),
        "dflash_verify": (i32, [vp, vp, i32, i32, vp, vp, vp]),
        "dflash_select_verify": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]),
        "dflash_lmhead_topk_static": (i32, [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp]),
        "dflash_gemm_bf16": (i32, [vp, vp, vp, i32, i32, i32, vp]),
        "dflash_conv2tap_dynamic_workspace": (sz, [i32, i32, i32]),
        "dflash_conv2tap_dynamic": (i32, [vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, sz, vp]),
        "dflash_path_walk": (i32, [vp, vp, vp, vp, vp, vp, ctypes.c_float, i32, i32, i32, i32, i32,
                                   vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "dflash_verify_rejection_workspace": (sz, [i32, i32, i32]),
        "dflash_lmhead_topk_records": (i32, [i32, i32, i32]),
        "dflash_lmhead_topk_partial": (i32, [vp, vp, i32, i32, i32, i32, vp, sz, vp, vp]),
        "dflash_lmhead_topk_merge": (i32, [vp, i32, i32, i32, i32, vp, vp, vp, vp]),
        "dflash_ctx_table": (i32, [vp, vp, i32, i32, i32, vp, vp]),
        "dflash_ctx_gate": (i32, [vp, vp, i32, i32, i32, vp, vp]),
        "dflash_ctx_walk": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, ctypes.c_float,
                                  vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "dflash_rmsnorm": (i32, [vp, vp, vp, ctypes.c_float, i32, i32, vp, vp, vp]),
        "dflash_rmsnorm_i8": (i32, [vp, vp, vp, ctypes.c_float, i32, i32, vp, vp, vp, vp]),
        "dflash_quant_i8": (i32, [vp, i32, i32, vp, vp, vp]),
        "dflash_gemm_i8": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp]),
        "dflash_token_logprobs": (i32, [vp, i32, ctypes.c_longlong, i32, i32, vp, ctypes.c_float, i32,
                                        vp, vp, vp, vp, vp, vp, vp, vp]),
        "dflash_emitted_logprobs": (i32, [vp, i32, ctypes.c_longlong, i32, i32, i32, vp, vp, vp, ctypes.c_float, i32,
                                          vp, vp, vp, vp, vp, vp, vp, vp]),
        "dflash_verify_rejection": (i32, [vp, ctypes.c_float, vp, vp, vp, vp, vp, vp, i32, i32, i32,
                                          vp, vp, vp, sz, vp, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _check_build_id(lib)
    return lib


def _check_build_id(lib):
    """Refuse a library compiled from other sources than the ones beside it
    (when the sources are present): stale native code must not pass for the
    current code."""
    build_py = os.path.join(os.path.dirname(LIB_PATH), "build.py")
    if not os.path.isdir(os.path.join(os.path.dirname(LIB_PATH), "csrc")) or not os.path.exists(build_py):
        return
    import importlib.util
    spec = importlib.util.spec_from_file_location("_dflash_build_check", build_py)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    have, want = lib.dflash_build_id().decode(), mod.source_hash()
    if have != want:
        raise ImportError(f"{LIB_PATH} was built from other sources (build id {have}, sources {want}): "
                          "rebuild it with `python block_draft_selection_b200/build.py`")


lib = _load()


def dflash_status_string(code: int) -> str:
    return lib.dflash_status_string(int(code)).decode()


def dflash_build_id() -> str:
    return lib.dflash_build_id().decode()


def _check(fn: str, code: int):
    if code != DFLASH_OK:
        raise DFlashError(fn, code)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _out(t, name, dtype, shape, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _need(t, name, dtype, shape)


def dflash_conv2tap(x, a0, a1, prev=None, y=None, stream=None):
    """y[b,t,c] = a0[c] x[b,t,c] + a1[c] x[b,t-1,c], x[b,-1,:] = prev[b,:] (zeros if None).
    x [B,P,d] bf16; a0, a1 [d] bf16; prev [B,d] bf16 or None."""
    _need(x, "x", torch.bfloat16)
    B, P, d = x.shape
    _need(a0, "a0", torch.bfloat16, (d,))
    _need(a1, "a1", torch.bfloat16, (d,))
    if prev is not None:
        _need(prev, "prev", torch.bfloat16, (B, d))
    y = _out(y, "y", torch.bfloat16, (B, P, d), x.device)
    _check("dflash_conv2tap", lib.dflash_conv2tap(_ptr(x), _ptr(prev), _ptr(a0), _ptr(a1), _ptr(y),
                                                  B, P, d, _stream(stream)))
    return y


def dflash_gemm_bf16(A, B, C=None, stream=None):
    """C [M,N] fp32 = A [M,K] bf16 . B [N,K]^T, on the tensor-core path."""
    _need(A, "A", torch.bfloat16)
    _need(B, "B", torch.bfloat16)
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K:
        raise ValueError("A and B disagree on K")
    C = _out(C, "C", torch.float32, (M, N), A.device)
    _check("dflash_gemm_bf16", lib.dflash_gemm_bf16(_ptr(A), _ptr(B), _ptr(C), M, N, K, _stream(stream)))
    return C


def dflash_conv2tap_dynamic_workspace(B: int, P: int, d: int) -> int:
    return int(lib.dflash_conv2tap_dynamic_workspace(B, P, d))


def dflash_conv2tap_dynamic(x, a0, a1, wc, prev=None, y=None, ws=None, stream=None):
    """Two-tap conv with per-16-channel tap corrections delta = x . Wc^T.
    x [B,P,d], a0/a1 [d], wc [2*d/16, d], prev [B,d] or None: bf16."""
    _need(x, "x", torch.bfloat16)
    B, P, d = x.shape
    _need(a0, "a0", torch.bfloat16, (d,))
    _need(a1, "a1", torch.bfloat16, (d,))
    _need(wc, "wc", torch.bfloat16, (2 * (d // 16), d))
    if prev is not None:
        _need(prev, "prev", torch.bfloat16, (B, d))
    y = _out(y, "y", torch.bfloat16, (B, P, d), x.device)
    if ws is None:
        n = dflash_conv2tap_dynamic_workspace(B, P, d)
        if n == 0:
            raise DFlashError("dflash_conv2tap_dynamic_workspace", DFLASH_ERR_INVALID_ARG)
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    _check("dflash_conv2tap_dynamic", lib.dflash_conv2tap_dynamic(
        _ptr(x), _ptr(prev), _ptr(a0), _ptr(a1), _ptr(wc), _ptr(y), B, P, d, _ptr(ws), ws.numel(),
        _stream(stream)))
    return y


def dflash_lmhead_topk_workspace(M: int, V: int, d: int) -> int:
    return int(lib.dflash_lmhead_topk_workspace(M, V, d))


def workspace(M: int, V: int, d: int, device="cuda") -> torch.Tensor:
    n = dflash_lmhead_topk_workspace(M, V, d)
    if n == 0:
        raise DFlashError("dflash_lmhead_topk_workspace", DFLASH_ERR_INVALID_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device)


def dflash_lmhead_topk(H, W, K=K_TOP, topk_logp=None, topk_idx=None, lse=None, ws=None,
                       dev_status=None, stream=None, want_lse=True):
    """H [M,d] bf16, W [V,d] bf16 -> (topk_logp [M,16] f32, topk_idx [M,16] i32, lse [M] f32)."""
    _need(H, "H", torch.bfloat16)
    _need(W, "W", torch.bfloat16)
    M, d = H.shape
    V = W.shape[0]
    if W.shape[1] != d:
        raise ValueError("H and W disagree on d")
    topk_logp = _out(topk_logp, "topk_logp", torch.float32, (M, K), H.device)
    topk_idx = _out(topk_idx, "topk_idx", torch.int32, (M, K), H.device)
    if lse is None and want_lse:
        lse = torch.empty(M, dtype=torch.float32, device=H.device)
    elif lse is not None:
        _need(lse, "lse", torch.float32, (M,))
    if ws is None:
        ws = workspace(M, V, d, H.device)
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, (1,))
    _check("dflash_lmhead_topk", lib.dflash_lmhead_topk(
        _ptr(H), _ptr(W), M, V, d, K, _ptr(topk_logp), _ptr(topk_idx), _ptr(lse), _ptr(ws),
        ws.numel(), _ptr(dev_status), _stream(stream)))
    return topk_logp, topk_idx, lse


def dflash_lmhead_logits_debug(H, W, z=None, ws=None, dev_status=None, stream=None):
    """Raw logits z [M,V] f32 through the same GEMM path (diagnostic)."""
    _need(H, "H", torch.bfloat16)
    _need(W, "W", torch.bfloat16)
    M, d = H.shape
    V = W.shape[0]
    z = _out(z, "z", torch.float32, (M, V), H.device)
    if ws is None:
        ws = workspace(M, V, d, H.device)
    _check("dflash_lmhead_logits_debug", lib.dflash_lmhead_logits_debug(
        _ptr(H), _ptr(W), M, V, d, _ptr(z), _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream)))
    return z


def dflash_path_select(topk_logp, topk_idx, E, Msel, B, L, path_tok=None, path_slot=None,
                       path_score=None, pair_scores=False, dev_status=None, stream=None):
    """Returns (path_tok [B,L] i32, path_slot [B,L] i32, path_score [B] f32, pair scores
    [B,L-1,16,16] f32 or None)."""
    _need(topk_logp, "topk_logp", torch.float32, (B * L, K_TOP))
    _need(topk_idx, "topk_idx", torch.int32, (B * L, K_TOP))
    _need(E, "E", torch.bfloat16)
    V, r = E.shape
    _need(Msel, "Msel", torch.bfloat16, (r, r))
    dev = topk_logp.device
    path_tok = _out(path_tok, "path_tok", torch.int32, (B, L), dev)
    path_slot = _out(path_slot, "path_slot", torch.int32, (B, L), dev)
    path_score = _out(path_score, "path_score", torch.float32, (B,), dev)
    pair = torch.empty((B, max(L - 1, 0), K_TOP, K_TOP), dtype=torch.float32, device=dev) if pair_scores else None
    _check("dflash_path_select", lib.dflash_path_select(
        _ptr(topk_logp), _ptr(topk_idx), _ptr(E), _ptr(Msel), B, L, K_TOP, r, V, _ptr(path_tok),
        _ptr(path_slot), _ptr(path_score), _ptr(pair) if pair is not None and pair.numel() else None,
        _ptr(dev_status), _stream(stream)))
    return path_tok, path_slot, path_score, pair


def dflash_select_verify(topk_logp, topk_idx, E, Msel, target, B, L, path_tok=None, path_slot=None,
                         path_score=None, accept_len=None, next_token=None, dev_status=None, stream=None):
    """Path selection and greedy verification of the chosen path in one kernel.
    Returns (path_tok, path_slot, path_score, accept_len, next_token)."""
    _need(topk_logp, "topk_logp", torch.float32, (B * L, K_TOP))
    _need(topk_idx, "topk_idx", torch.int32, (B * L, K_TOP))
    _need(E, "E", torch.bfloat16)
    V, r = E.shape
    _need(Msel, "Msel", torch.bfloat16, (r, r))
    _need(target, "target", torch.int32, (B, L + 1))
    dev = topk_logp.device
    path_tok = _out(path_tok, "path_tok", torch.int32, (B, L), dev)
    path_slot = _out(path_slot, "path_slot", torch.int32, (B, L), dev)
    path_score = _out(path_score, "path_score", torch.float32, (B,), dev)
    accept_len = _out(accept_len, "accept_len", torch.int32, (B,), dev)
    next_token = _out(next_token, "next_token", torch.int32, (B,), dev)
    _check("dflash_select_verify", lib.dflash_select_verify(
        _ptr(topk_logp), _ptr(topk_idx), _ptr(E), _ptr(Msel), _ptr(target), B, L, K_TOP, r, V,
        _ptr(path_tok), _ptr(path_slot), _ptr(path_score), _ptr(accept_len), _ptr(next_token),
        _ptr(dev_status), _stream(stream)))
    return path_tok, path_slot, path_score, accept_len, next_token


def dflash_lmhead_topk_static(H, W, K=K_TOP, topk_logp=None, topk_idx=None, lse=None, dev_status=None,
                              stream=None):
    """dflash_lmhead_topk without a workspace (library-owned scratch; see the header)."""
    _need(H, "H", torch.bfloat16)
    _need(W, "W", torch.bfloat16)
    M, d = H.shape
    V = W.shape[0]
    topk_logp = _out(topk_logp, "topk_logp", torch.float32, (M, K), H.device)
    topk_idx = _out(topk_idx, "topk_idx", torch.int32, (M, K), H.device)
    lse = _out(lse, "lse", torch.float32, (M,), H.device)
    _check("dflash_lmhead_topk_static", lib.dflash_lmhead_topk_static(
        _ptr(H), _ptr(W), M, V, d, K, _ptr(topk_logp), _ptr(topk_idx), _ptr(lse), _ptr(dev_status),
        _stream(stream)))
    return topk_logp, topk_idx, lse


def dflash_verify(draft, target, accept_len=None, next_token=None, stream=None):
    """draft [B,L] i32, target [B,L+1] i32 -> (accept_len [B] i32, next_token [B] i32)."""
    _need(draft, "draft", torch.int32)
    B, L = draft.shape
    _need(target, "target", torch.int32, (B, L + 1))
    accept_len = _out(accept_len, "accept_len", torch.int32, (B,), draft.device)
    next_token = _out(next_token, "next_token", torch.int32, (B,), draft.device)
    _check("dflash_verify", lib.dflash_verify(_ptr(draft), _ptr(target), B, L, _ptr(accept_len),
                                              _ptr(next_token), _stream(stream)))
    return accept_len, next_token


def dflash_path_walk(topk_logp, topk_idx, E, Msel, anchor, B, L, uniforms=None, temperature=1.0,
                     path_tok=None, path_slot=None, path_score=None, path_q=None, want_q=True,
                     target=None, accept_len=None, next_token=None, dev_status=None, stream=None):
    """Walk from the last verified token: greedy when `uniforms` is None, else sampled
    at `temperature`.  Returns (path_tok, path_slot, path_score, path_q or None,
    accept_len or None, next_token or None); the last two only when `target` is given."""
    _need(topk_logp, "topk_logp", torch.float32, (B * L, K_TOP))
    _need(topk_idx, "topk_idx", torch.int32, (B * L, K_TOP))
    _need(E, "E", torch.bfloat16)
    V, r = E.shape
    _need(Msel, "Msel", torch.bfloat16, (r, r))
    _need(anchor, "anchor", torch.int32, (B,))
    dev = topk_logp.device
    if uniforms is not None:
        _need(uniforms, "uniforms", torch.float32, (B, L))
    path_tok = _out(path_tok, "path_tok", torch.int32, (B, L), dev)
    path_slot = _out(path_slot, "path_slot", torch.int32, (B, L), dev)
    path_score = _out(path_score, "path_score", torch.float32, (B,), dev)
    if uniforms is not None and (want_q or path_q is not None):
        path_q = _out(path_q, "path_q", torch.float32, (B, L, K_TOP), dev)
    else:
        path_q = None
    if target is not None:
        _need(target, "target", torch.int32, (B, L + 1))
        accept_len = _out(accept_len, "accept_len", torch.int32, (B,), dev)
        next_token = _out(next_token, "next_token", torch.int32, (B,), dev)
    else:
        accept_len = next_token = None
    _check("dflash_path_walk", lib.dflash_path_walk(
        _ptr(topk_logp), _ptr(topk_idx), _ptr(E), _ptr(Msel), _ptr(anchor), _ptr(uniforms),
        float(temperature), B, L, K_TOP, r, V, _ptr(path_tok), _ptr(path_slot), _ptr(path_score),
        _ptr(path_q), _ptr(target), _ptr(accept_len), _ptr(next_token), _ptr(dev_status), _stream(stream)))
    return path_tok, path_slot, path_score, path_q, accept_len, next_token


def dflash_verify_rejection_workspace(B: int, L: int, V: int) -> int:
    return int(lib.dflash_verify_rejection_workspace(B, L, V))


def dflash_verify_rejection(target_logits, temperature, draft, draft_slot, cand_idx, draft_q, u_accept,
                            u_resample, accept_len=None, next_token=None, ws=None, dev_status=None,
                            stream=None):
    """Rejection-sampling verification.  target_logits [B*(L+1), V] f32; draft, draft_slot
    [B, L] i32; cand_idx [B*L, 16] i32; draft_q [B, L, 16] f32; u_accept [B, L] f32;
    u_resample [B] f32.  Returns (accept_len [B] i32, next_token [B] i32)."""
    _need(draft, "draft", torch.int32)
    B, L = draft.shape
    _need(target_logits, "target_logits", torch.float32)
    V = target_logits.shape[1]
    _need(target_logits, "target_logits", torch.float32, (B * (L + 1), V))
    _need(draft_slot, "draft_slot", torch.int32, (B, L))
    _need(cand_idx, "cand_idx", torch.int32, (B * L, K_TOP))
    _need(draft_q, "draft_q", torch.float32, (B, L, K_TOP))
    _need(u_accept, "u_accept", torch.float32, (B, L))
    _need(u_resample, "u_resample", torch.float32, (B,))
    dev = draft.device
    accept_len = _out(accept_len, "accept_len", torch.int32, (B,), dev)
    next_token = _out(next_token, "next_token", torch.int32, (B,), dev)
    if ws is None:
        ws = torch.empty(max(16, dflash_verify_rejection_workspace(B, L, V)), dtype=torch.uint8, device=dev)
    _check("dflash_verify_rejection", lib.dflash_verify_rejection(
        _ptr(target_logits), float(temperature), _ptr(draft), _ptr(draft_slot), _ptr(cand_idx),
        _ptr(draft_q), _ptr(u_accept), _ptr(u_resample), B, L, V, _ptr(accept_len), _ptr(next_token),
        _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream)))
    return accept_len, next_token


def dflash_ctx_table(Emb, Pab, tab=None, stream=None):
    """A and B of the context-gated scorer for every token: tab [V, 2e] fp32
    = Emb . Pab^T (row v: A(v), then B(v)).  Computed once per weight set."""
    _need(Emb, "Emb", torch.bfloat16)
    V, d = Emb.shape
    _need(Pab, "Pab", torch.bfloat16)
    e = Pab.shape[0] // 2
    _need(Pab, "Pab", torch.bfloat16, (2 * e, d))
    tab = _out(tab, "tab", torch.float32, (V, 2 * e), Emb.device)
    _check("dflash_ctx_table", lib.dflash_ctx_table(_ptr(Emb), _ptr(Pab), V, d, e, _ptr(tab), _stream(stream)))
    return tab


def dflash_ctx_gate(H, Pg, gate=None, stream=None):
    """The context gate before its sigmoid: gate [M, e] fp32 = H . Pg^T."""
    _need(H, "H", torch.bfloat16)
    M, d = H.shape
    _need(Pg, "Pg", torch.bfloat16)
    e = Pg.shape[0]
    _need(Pg, "Pg", torch.bfloat16, (e, d))
    gate = _out(gate, "gate", torch.float32, (M, e), H.device)
    _check("dflash_ctx_gate", lib.dflash_ctx_gate(_ptr(H), _ptr(Pg), M, d, e, _ptr(gate), _stream(stream)))
    return gate


_WALKS = {"maxsum": 0, "greedy": 1, "sample": 2}


def dflash_ctx_walk(topk_logp, topk_idx, anchor, tab, gate, B, L, V, walk="maxsum", uniforms=None,
                    temperature=1.0, want_tables=False, target=None, path_tok=None, path_slot=None,
                    path_score=None, path_q=None, accept_len=None, next_token=None, dev_status=None, stream=None):
    """Scores of the context-gated scorer and a walk from the anchor.  Returns
    (path_tok, path_slot, path_score, path_q or None, tables or None,
    accept_len or None, next_token or None)."""
    _need(topk_logp, "topk_logp", torch.float32, (B * L, K_TOP))
    _need(topk_idx, "topk_idx", torch.int32, (B * L, K_TOP))
    _need(anchor, "anchor", torch.int32, (B,))
    _need(gate, "gate", torch.float32)
    e = gate.shape[1]
    _need(gate, "gate", torch.float32, (B * L, e))
    _need(tab, "tab", torch.float32, (V, 2 * e))
    dev = tab.device
    if walk == "sample":
        _need(uniforms, "uniforms", torch.float32, (B, L))
    path_tok = _out(path_tok, "path_tok", torch.int32, (B, L), dev)
    path_slot = _out(path_slot, "path_slot", torch.int32, (B, L), dev)
    path_score = _out(path_score, "path_score", torch.float32, (B,), dev)
    path_q = _out(path_q, "path_q", torch.float32, (B, L, K_TOP), dev) if walk == "sample" else None
    tables = torch.empty((B, L, K_TOP, K_TOP), dtype=torch.float32, device=dev) if want_tables else None
    if target is not None:
        _need(target, "target", torch.int32, (B, L + 1))
        accept_len = _out(accept_len, "accept_len", torch.int32, (B,), dev)
        next_token = _out(next_token, "next_token", torch.int32, (B,), dev)
    else:
        accept_len = next_token = None
    _check("dflash_ctx_walk", lib.dflash_ctx_walk(
        _ptr(topk_logp), _ptr(topk_idx), _ptr(anchor), _ptr(tab), _ptr(gate), B, L, K_TOP, e, V, _WALKS[walk],
        _ptr(uniforms) if walk == "sample" else None, float(temperature), _ptr(path_tok), _ptr(path_slot),
        _ptr(path_score), _ptr(path_q), _ptr(tables), _ptr(target), _ptr(accept_len), _ptr(next_token),
        _ptr(dev_status), _stream(stream)))
    return path_tok, path_slot, path_score, path_q, tables, accept_len, next_token


RECORD_WORDS = 36   # one partial record: max, sum, 2 unused, 16 values, 16 indices


def dflash_lmhead_topk_records(M: int, V: int, d: int) -> int:
    return int(lib.dflash_lmhead_topk_records(M, V, d))


def dflash_lmhead_topk_partial(H, W, v_offset=0, records=None, dev_status=None, stream=None):
    """Partial records [M, P, 36] (float32 words) of H . W^T over this shard of
    the head, vocabulary indices shifted by v_offset."""
    _need(H, "H", torch.bfloat16)
    _need(W, "W", torch.bfloat16)
    M, d = H.shape
    V = W.shape[0]
    P = dflash_lmhead_topk_records(M, V, d)
    if P <= 0:
        raise DFlashError("dflash_lmhead_topk_records", DFLASH_ERR_INVALID_ARG)
    records = _out(records, "records", torch.float32, (M, P, RECORD_WORDS), H.device)
    _check("dflash_lmhead_topk_partial", lib.dflash_lmhead_topk_partial(
        _ptr(H), _ptr(W), M, V, d, int(v_offset), _ptr(records), records.numel() * 4, _ptr(dev_status),
        _stream(stream)))
    return records


def dflash_lmhead_topk_merge(records, topk_logp=None, topk_idx=None, lse=None, stream=None):
    """records [nrank, M, P, 36] float32 -> (topk_logp [M,16], topk_idx [M,16], lse [M])."""
    _need(records, "records", torch.float32)
    if records.dim() == 3:
        records = records.unsqueeze(0)
    nrank, M, P, w = records.shape
    if w != RECORD_WORDS:
        raise ValueError("records must have 36 words per record")
    topk_logp = _out(topk_logp, "topk_logp", torch.float32, (M, K_TOP), records.device)
    topk_idx = _out(topk_idx, "topk_idx", torch.int32, (M, K_TOP), records.device)
    lse = _out(lse, "lse", torch.float32, (M,), records.device)
    _check("dflash_lmhead_topk_merge", lib.dflash_lmhead_topk_merge(
        _ptr(records), M, P, nrank, K_TOP, _ptr(topk_logp), _ptr(topk_idx), _ptr(lse), _stream(stream)))
    return topk_logp, topk_idx, lse


# ---- the operators around a cycle: norm, int8, log-probabilities ----------
#
# These check that every tensor is on one device, launch on that device
# whichever one is current, and allocate what the caller did not pass on the
# stream they launch on.

def _arg(t, name, dtype, shape, index):
    """The device pointer of a contiguous CUDA tensor of this type, shape and device."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        return t.data_ptr()
    _need(t, name, dtype, shape)
    raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _on(stream, index):
    """The stream to launch on, as an integer."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    if stream.device_index != index:
        raise ValueError(f"stream must be on cuda:{index}, got cuda:{stream.device_index}")
    return stream.cuda_stream


def _empty(shape, dtype, device):
    # with its strides given: 1.5 us a call instead of torch.empty's 2.4
    return torch.empty_strided(shape, (1,) if len(shape) == 1 else (shape[1], 1), dtype=dtype, device=device)


def _new(dtype, shape, index, stream, make=_empty):
    if stream is None:
        return make(shape, dtype=dtype, device=index)
    with torch.cuda.stream(stream):   # so that the allocator ties the memory to the stream that uses it
        return make(shape, dtype=dtype, device=index)


def _call(name, index, *args):
    """Call the entry point with the tensors' device current."""
    if torch._C._cuda_getDevice() == index:
        code = _FN[name](*args)
    else:
        with torch.cuda.device(index):
            code = _FN[name](*args)
    if code != DFLASH_OK:
        raise DFlashError(name, code)


_FN = {n: getattr(lib, n) for n in ("dflash_rmsnorm", "dflash_rmsnorm_i8", "dflash_quant_i8", "dflash_gemm_i8",
                                    "dflash_token_logprobs", "dflash_emitted_logprobs")}


def _matrix(t, name, dtype):
    """Shape, device and pointer of a contiguous CUDA matrix of this type."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        _need(t, name, dtype)
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    return t.shape, t.get_device(), t.data_ptr()


def _given_or_new(t, name, dtype, shape, index, stream):
    """An output and its pointer."""
    if t is None:
        t = _new(dtype, shape, index, stream)
        return t, t.data_ptr()
    return t, _arg(t, name, dtype, shape, index)


def _norm_inputs(x, gamma, residual, h, stream):
    """(M, d, device index, pointers of x, residual, gamma and h, h)."""
    shape, index, px = _matrix(x, "x", torch.bfloat16)
    M, d = shape
    pg = _arg(gamma, "gamma", torch.bfloat16, (d,), index)
    if residual is None:
        if h is not None:
            raise ValueError("h is the sum with a residual: there is none")
        return M, d, index, px, None, pg, None, None
    pr = _arg(residual, "residual", torch.bfloat16, shape, index)
    h, ph = _given_or_new(h, "h", torch.bfloat16, shape, index, stream)
    return M, d, index, px, pr, pg, ph, h


def dflash_rmsnorm(x, gamma, residual=None, eps=1e-6, y=None, h=None, stream=None):
    """h = bf16(x + residual) (x without one), y = h * gamma / sqrt(mean h^2 + eps).
    x, residual [M,d], gamma [d] bf16 -> (y [M,d] bf16, h [M,d] bf16 or None without a residual).
    h and y may each be x or residual (an update in place), not each other."""
    M, d, index, px, pr, pg, ph, h = _norm_inputs(x, gamma, residual, h, stream)
    y, py = _given_or_new(y, "y", torch.bfloat16, (M, d), index, stream)
    _call("dflash_rmsnorm", index, px, pr, pg, eps, M, d, ph, py, _on(stream, index))
    return y, h


def dflash_rmsnorm_i8(x, gamma, residual=None, eps=1e-6, q=None, scale=None, h=None, stream=None):
    """dflash_rmsnorm with its output in int8 and a scale per row (q * scale is the normalised row):
    (q [M,d] int8, scale [M] f32, h [M,d] bf16 or None without a residual)."""
    M, d, index, px, pr, pg, ph, h = _norm_inputs(x, gamma, residual, h, stream)
    q, pq = _given_or_new(q, "q", torch.int8, (M, d), index, stream)
    scale, ps = _given_or_new(scale, "scale", torch.float32, (M,), index, stream)
    _call("dflash_rmsnorm_i8", index, px, pr, pg, eps, M, d, ph, pq, ps, _on(stream, index))
    return q, scale, h


def dflash_quant_i8(x, q=None, scale=None, stream=None):
    """Rows x [M,d] bf16 -> (q [M,d] int8, scale [M] f32 = max|row| / 127)."""
    shape, index, px = _matrix(x, "x", torch.bfloat16)
    M, d = shape
    q, pq = _given_or_new(q, "q", torch.int8, shape, index, stream)
    scale, ps = _given_or_new(scale, "scale", torch.float32, (M,), index, stream)
    _call("dflash_quant_i8", index, px, M, d, pq, ps, _on(stream, index))
    return q, scale


def dflash_gemm_i8(A, sa, B, sb, C=None, dtype=torch.float32, dev_status=None, stream=None):
    """C [M,N] = (A [M,K] int8 . B [N,K]^T int8, exact in int32) * sa [M] * sb [N]; C in f32 or bf16
    (`dtype`, or C's own type)."""
    (M, K), index, pa = _matrix(A, "A", torch.int8)
    (N, Kb), index_b, pb = _matrix(B, "B", torch.int8)
    if Kb != K:
        raise ValueError("A and B disagree on K")
    if index_b != index:
        raise ValueError(f"B must be on cuda:{index}, got {B.device}")
    if C is not None:
        dtype = C.dtype
    if dtype is not torch.float32 and dtype is not torch.bfloat16:
        raise TypeError(f"C must be {torch.float32} or {torch.bfloat16}, got {dtype}")
    C, pc = _given_or_new(C, "C", dtype, (M, N), index, stream)
    _call("dflash_gemm_i8", index, pa, _arg(sa, "sa", torch.float32, (M,), index), pb,
          _arg(sb, "sb", torch.float32, (N,), index), pc, 1 if dtype is torch.bfloat16 else 0, M, N, K,
          _status(dev_status, index), _on(stream, index))
    return C


def _status(dev_status, index):
    return None if dev_status is None else _arg(dev_status, "dev_status", torch.int32, (1,), index)


def _logits(z, name):
    """(pointer, is bf16, row stride, rows, V, device index) of a matrix of logits whose rows are contiguous."""
    if not isinstance(z, torch.Tensor) or not z.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if z.dtype is not torch.float32 and z.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.float32} or {torch.bfloat16}, got {z.dtype}")
    if z.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {z.dim()}")
    rows, V = z.shape
    ld, step = z.stride()
    if rows == 1:
        ld = V
    if (V > 1 and step != 1) or ld < V:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return z.data_ptr(), 1 if z.dtype is torch.bfloat16 else 0, ld, rows, V, z.get_device()


def _logprob_out(t, name, dtype, shape, index, stream):
    """An output and its pointer.  What the call allocates is zeroed: rows that are not asked for are not written."""
    if t is None:
        t = _new(dtype, shape, index, stream, torch.zeros)
    return t, _arg(t, name, dtype, shape, index)


def _logprob_outs(shape, K, index, stream, logp, rank, entropy, lse, top_logp, top_idx, with_token=True):
    """Outputs in the order logp, rank, entropy, lse, top_logp, top_idx, and their pointers."""
    if not 0 <= K <= 32:
        raise ValueError(f"K must be in [0, 32], got {K}")
    f32, i32 = torch.float32, torch.int32
    if with_token and logp is rank is entropy is lse is top_logp is top_idx is None:
        # none given: parts of one buffer, zeroed by one launch instead of six
        n = math.prod(shape)
        flat = _new(f32, (n * (4 + 2 * K),), index, stream, torch.zeros)
        logp, rank, entropy, lse, top_logp, top_idx = flat.split((n, n, n, n, n * K, n * K))
        outs = (logp, rank.view(i32), entropy, lse, top_logp.view(*shape, K), top_idx.view(i32).view(*shape, K))
        if len(shape) > 1:
            outs = (*(t.view(shape) for t in outs[:4]), *outs[4:])
        p = flat.data_ptr()
        ptrs = tuple(p + 4 * n * i for i in (0, 1, 2, 3, 4, 4 + K))
        return outs, ptrs if K else (*ptrs[:4], None, None)
    if with_token:
        logp, p0 = _logprob_out(logp, "logp", f32, shape, index, stream)
        rank, p1 = _logprob_out(rank, "rank", i32, shape, index, stream)
    elif logp is not None or rank is not None:
        raise ValueError("logp and rank need tokens")
    else:
        p0 = p1 = None
    entropy, p2 = _logprob_out(entropy, "entropy", f32, shape, index, stream)
    lse, p3 = _logprob_out(lse, "lse", f32, shape, index, stream)
    top = (*shape, K)
    top_logp, p4 = _logprob_out(top_logp, "top_logp", f32, top, index, stream)
    top_idx, p5 = _logprob_out(top_idx, "top_idx", i32, top, index, stream)
    if K == 0:
        p4 = p5 = None
    return (logp, rank, entropy, lse, top_logp, top_idx), (p0, p1, p2, p3, p4, p5)


def dflash_token_logprobs(logits, tokens=None, K=K_TOP, temperature=1.0, logp=None, rank=None, entropy=None, lse=None,
                          top_logp=None, top_idx=None, dev_status=None, stream=None):
    """Log-probabilities of one given token per row of logits [M,V] (f32 or bf16; rows may be strided), with the
    token's rank, the row's entropy and log-sum-exp, and its K best tokens.  tokens [M] i32 (negative: the row is
    not asked for, its outputs stay as they are) or None.  Returns (logp [M], rank [M] i32, entropy [M], lse [M],
    top_logp [M,K], top_idx [M,K] i32); logp and rank are None without tokens.  With tokens and no output given, all of
    them are parts of one buffer: keeping or saving one keeps or saves all (clone() it, or pass outputs)."""
    pz, z_bf16, ld, M, V, index = _logits(logits, "logits")
    pt = None if tokens is None else _arg(tokens, "tokens", torch.int32, (M,), index)
    outs, ptrs = _logprob_outs((M,), K, index, stream, logp, rank, entropy, lse, top_logp, top_idx, tokens is not None)
    _call("dflash_token_logprobs", index, pz, z_bf16, ld, M, V, pt, temperature, K, *ptrs,
          _status(dev_status, index), _on(stream, index))
    return outs


def dflash_emitted_logprobs(target_logits, draft, accept_len, next_token, K=K_TOP, temperature=1.0, logp=None,
                            rank=None, entropy=None, lse=None, top_logp=None, top_idx=None, dev_status=None,
                            stream=None):
    """dflash_token_logprobs for the tokens that a verification step emitted: draft [B,L], accept_len [B],
    next_token [B] i32 and the target_logits [B*(L+1),V] they were verified against.  Outputs [B,L+1] (and
    [B,L+1,K]); positions at and past accept_len stay as they are (zero where the call allocates).  With no output
    given, all of them are parts of one buffer, as dflash_token_logprobs says."""
    pz, z_bf16, ld, rows, V, index = _logits(target_logits, "target_logits")
    (B, L), _, pd = _matrix(draft, "draft", torch.int32)
    if rows != B * (L + 1):
        raise ValueError(f"target_logits must have {B * (L + 1)} rows, got {rows}")
    if draft.get_device() != index:
        raise ValueError(f"draft must be on cuda:{index}, got {draft.device}")
    pa = _arg(accept_len, "accept_len", torch.int32, (B,), index)
    pn = _arg(next_token, "next_token", torch.int32, (B,), index)
    outs, ptrs = _logprob_outs((B, L + 1), K, index, stream, logp, rank, entropy, lse, top_logp, top_idx)
    _call("dflash_emitted_logprobs", index, pz, z_bf16, ld, B, L, V, pd, pa, pn, temperature, K, *ptrs,
          _status(dev_status, index), _on(stream, index))
    return outs
