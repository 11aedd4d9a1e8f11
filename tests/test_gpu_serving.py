"""The norm, the int8 product and the log-probabilities together, as a serving
program runs them around a draft cycle, on streams and in CUDA graphs."""
import math

import numpy as np
import pytest
import torch

import oracle
import block_draft_synth as syn
from helpers import dev_bf16

pytestmark = pytest.mark.gpu


def _model(w):
    x, prev = syn.conv_input(w)
    rng = np.random.default_rng(w.seed)
    gamma = syn.f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(w.d)).astype(np.float32))
    return syn.hidden(w), syn.lm_head(w), gamma


def _quantised_logits(H, res, gamma, Wq, sw):
    """The oracle's int8 head on the GPU's own bits: every step is exact or
    defined rounding but the scales, whose fp32 value is taken as given."""
    q, scale, h = oracle.rmsnorm_i8(H, gamma, res)
    return q, scale, h


@pytest.mark.parametrize("name", ["tiny", "qwen3-4b-bs1"])
def test_int8_head_of_the_drafter(name):
    """norm with residual -> int8 -> product with the quantised head -> top-16
    and lse -> path selection and verification: every stage against the
    oracle's on that stage's inputs, and the candidates against the bf16
    head's."""
    import block_draft_selection_b200 as bds
    w = syn.workload(name)
    H, W, gamma = _model(w)
    res = syn.hidden(syn.Workload(w.name, B=w.B, L=w.L, P=w.P, d=w.d, V=w.V, r=w.r, sigma=w.sigma, seed=w.seed + 50))
    E, Msel = syn.selector_tables(w)
    Wd = dev_bf16(W)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Wq, sw = bds.dflash_quant_i8(Wd)
    q, sh, h = bds.dflash_rmsnorm_i8(dev_bf16(H), dev_bf16(gamma), residual=dev_bf16(res))
    z = bds.dflash_gemm_i8(q, sh, Wq, sw, dev_status=status)
    _, _, ent, lse, lp, ix = bds.dflash_token_logprobs(z, K=16, dev_status=status)
    tok, slot, score, _ = bds.dflash_path_select(lp, ix, dev_bf16(E), dev_bf16(Msel), w.B, w.L, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    qr, shr, _ = oracle.rmsnorm_i8(H, gamma, res)
    np.testing.assert_array_equal(q.cpu().numpy(), qr)
    rows = np.random.default_rng(0).choice(w.V, 2000, replace=False)
    wq, swr = oracle.quant_i8(W[rows])
    np.testing.assert_array_equal(Wq[torch.from_numpy(rows).cuda()].cpu().numpy(), wq)
    zr = oracle.gemm_i8(qr, sh.cpu().numpy(), wq, swr.astype(np.float32))
    np.testing.assert_array_equal(z[:, torch.from_numpy(rows).cuda()].cpu().numpy(), zr)
    ref = oracle.token_logprobs(z.double().cpu().numpy(), np.zeros(w.M, int), 1.0, 16)
    np.testing.assert_array_equal(ix.cpu().numpy(), ref["top_idx"])
    assert np.abs(lp.double().cpu().numpy() - ref["top_logp"]).max() < 1e-5
    path = oracle.path_select(lp.cpu().numpy(), ix.cpu().numpy(), E, Msel, w.B, w.L)
    firm = path["margin"] >= 1e-3
    np.testing.assert_array_equal(tok.cpu().numpy()[firm], path["path_tok"][firm])
    # and the 8-bit head stands for the bf16 one: the step of a logit is about
    # sqrt(d) * step(h) * step(w) / sqrt(12) ~ 1% of its spread, so the best
    # token is among the other's 16
    y, _ = bds.dflash_rmsnorm(dev_bf16(H), dev_bf16(gamma), residual=dev_bf16(res))
    _, ix16, _ = bds.dflash_lmhead_topk(y, Wd)
    torch.cuda.synchronize()
    a, b = ix.cpu().numpy(), ix16.cpu().numpy()
    assert all(b[m, 0] in a[m] and a[m, 0] in b[m] for m in range(w.M))


def _verification(B, L, V, d, seed):
    """A sampled draft and a target whose logits come from the int8 head."""
    import block_draft_selection_b200 as bds
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    s = {"x": rnd(B * (L + 1), d).bfloat16(), "res": rnd(B * (L + 1), d).bfloat16(), "gamma": (2 + 0.1 * rnd(d)).bfloat16()}
    s["Wq"], s["sw"] = bds.dflash_quant_i8((rnd(V, d) / math.sqrt(d)).bfloat16())
    idx = torch.stack([torch.randperm(V, generator=g, device="cuda")[:16] for _ in range(B * L)]).int()
    qd = torch.softmax(rnd(B, L, 16), dim=2)
    slot = torch.randint(0, 16, (B, L), generator=g, device="cuda", dtype=torch.int32)
    s |= {"idx": idx, "q": qd, "slot": slot,
          "draft": torch.gather(idx.view(B, L, 16), 2, slot.long()[..., None])[..., 0].contiguous(),
          "ua": torch.rand((B, L), generator=g, device="cuda") * 1e-4, "ur": torch.rand(B, generator=g, device="cuda")}
    return s


def _target_step(s, B, L, out=None):
    import block_draft_selection_b200 as bds
    q, sh, h = bds.dflash_rmsnorm_i8(s["x"], s["gamma"], residual=s["res"])
    z = bds.dflash_gemm_i8(q, sh, s["Wq"], s["sw"])
    acc, nxt = bds.dflash_verify_rejection(z, 1.0, s["draft"], s["slot"], s["idx"], s["q"], s["ua"], s["ur"])
    return z, acc, nxt, bds.dflash_emitted_logprobs(z, s["draft"], acc, nxt, K=20, **(out or {}))


def _check_step(s, z, acc, nxt, out, V):
    t = oracle.emitted_tokens(s["draft"].cpu().numpy(), acc.cpu().numpy(), nxt.cpu().numpy())
    ref = oracle.token_logprobs(z.double().cpu().numpy(), t, 1.0, 20)
    for k, name in enumerate(("logp", "rank", "entropy", "lse", "top_logp", "top_idx")):
        got = out[k].reshape(-1, *out[k].shape[2:]).cpu().numpy()
        if name in ("rank", "top_idx"):
            np.testing.assert_array_equal(got, ref[name])
        else:
            assert np.abs(got - ref[name]).max() < 2e-5, name


@pytest.mark.parametrize("B,L,V,d", [(1, 7, 40000, 256), (24, 5, 3001, 272), (40, 4, 2000, 144)])
def test_verification_step_with_logprobs(B, L, V, d):
    """norm -> int8 logits of the target -> rejection verification -> the emitted tokens' log-probabilities."""
    s = _verification(B, L, V, d, B + L)
    z, acc, nxt, out = _target_step(s, B, L)
    torch.cuda.synchronize()
    assert ((acc >= 1) & (acc <= L + 1)).all()
    _check_step(s, z, acc, nxt, out, V)


def test_verification_step_captured_and_replayed():
    """Two graphs of the step over the same weights, replayed on two streams
    at once with new inputs each time: equal to eager runs."""
    B, L, V, d = 8, 5, 9001, 256
    cases = [[_verification(B, L, V, d, 100 + 10 * g + k) for k in range(3)] for g in range(2)]
    live = [{k: v.clone() for k, v in c[0].items()} for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, results = [], []
    for s, st in zip(live, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            _target_step(s, B, L)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            results.append(_target_step(s, B, L))
        graphs.append(g)
    for k in range(3):
        torch.cuda.synchronize()
        for s, c in zip(live, cases):
            for name, t in c[k].items():
                s[name].copy_(t)
        torch.cuda.synchronize()
        for _ in range(3):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for c, (z, acc, nxt, out) in zip(cases, results):
            ez, ea, en, eo = _target_step(c[k], B, L)
            assert torch.equal(z, ez) and torch.equal(acc, ea) and torch.equal(nxt, en)
            keep = (torch.arange(L + 1, device="cuda")[None] < ea[:, None])
            for a, b in zip(out, eo):
                assert torch.equal(a[keep], b[keep])


def test_calls_follow_their_stream():
    """Inputs produced late on a side stream, passed as `stream`: the calls wait for them."""
    import block_draft_selection_b200 as bds
    side = torch.cuda.Stream()
    M, V, d = 64, 20000, 1024
    g = torch.Generator(device="cuda").manual_seed(0)
    x0 = torch.randn((M, d), generator=g, device="cuda").bfloat16()
    gamma = torch.ones(d, device="cuda").bfloat16()
    Wq, sw = bds.dflash_quant_i8(torch.randn((V, d), generator=g, device="cuda").bfloat16())
    big = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big = big @ big * 1e-2
        x = x0 * 1.0
    q, sh, _ = bds.dflash_rmsnorm_i8(x, gamma, stream=side)
    z = bds.dflash_gemm_i8(q, sh, Wq, sw, stream=side)
    out = bds.dflash_token_logprobs(z, K=16, stream=side)
    side.synchronize()
    q2, sh2, _ = bds.dflash_rmsnorm_i8(x0, gamma)
    z2 = bds.dflash_gemm_i8(q2, sh2, Wq, sw)
    out2 = bds.dflash_token_logprobs(z2, K=16)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(z, z2)
    assert all(torch.equal(a, b) for a, b in zip(out[2:], out2[2:]))
