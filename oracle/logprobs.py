"""Log-probabilities of given tokens, entropy, rank and top alternatives, float64.

p = softmax(z / T); logp = log p[t]; entropy = -sum p log p (0 log 0 = 0);
rank = 1 + #{v : z[v] > z[t]}; alternatives by value descending, then index
ascending.  A row with nothing but -inf has lse = -inf, log-probabilities
-inf and entropy 0.  The DFlash 2 pages have no counterpart; a serving program
answers with these for the tokens a verification step emits.
"""
import numpy as np


def row_logprobs(z, T=1.0):
    """(log p [V], lse, entropy) of one row."""
    y = np.asarray(z, dtype=np.float64) / T
    m = y.max()
    if m == -np.inf:
        return np.full(y.shape, -np.inf), -np.inf, 0.0
    e = np.exp(y - m)
    lse = m + np.log(e.sum())
    lp = (y - m) - np.log(e.sum())     # not y - lse: both may be near the type's lowest value
    p = e / e.sum()
    live = p > 0
    return lp, lse, float(-(p[live] * lp[live]).sum())


def token_logprobs(z, tokens, T=1.0, K=16):
    """z [M, V] float, tokens [M] (negative: row not asked for) -> dict of
    arrays; rows not asked for hold zeros."""
    M, V = z.shape
    out = {"logp": np.zeros(M), "rank": np.zeros(M, np.int64), "entropy": np.zeros(M), "lse": np.zeros(M),
           "top_logp": np.zeros((M, K)), "top_idx": np.zeros((M, K), np.int64)}
    for m in range(M):
        t = int(tokens[m])
        if t < 0:
            continue
        lp, lse, ent = row_logprobs(z[m], T)
        order = np.lexsort((np.arange(V), -np.asarray(z[m], dtype=np.float64)))[:K]
        out["logp"][m] = lp[t]
        out["rank"][m] = 1 + int((z[m] > z[m][t]).sum())
        out["entropy"][m] = ent
        out["lse"][m] = lse
        out["top_logp"][m] = lp[order]
        out["top_idx"][m] = order
    return out


def emitted_tokens(draft, accept_len, next_token):
    """Tokens of rows b*(L+1) + i; -1 for the rows behind the accepted ones."""
    B, L = draft.shape
    t = np.full((B, L + 1), -1, dtype=np.int64)
    for b in range(B):
        n = int(accept_len[b])
        t[b, :n - 1] = draft[b, :n - 1]
        t[b, n - 1] = next_token[b]
    return t.reshape(-1)
