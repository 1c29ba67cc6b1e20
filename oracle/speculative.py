"""fp64 definitions for drafted trees over the carried state of the causal recurrence (one head, or
one sequence, at a time).

The masked FA-part with the set J(i) of a node's ancestors and itself in place of j <= i, the
recurrence over several tokens, and the verification walk of speculative sampling with given random
numbers: accept a drafted token with probability min(1, w(x) / (Z q(x))), replace a rejected one's
distribution by the residual max(w - Z q, 0), so that the tokens that come out are distributed as
samples of the target. Pinned by ``tests/test_oracle_speculative.py`` against the single-token step
and by the emitted tokens' distribution.
"""

import numpy as np

from .favor import phi


def ancestors(parents, i):
    """Node i, its parent, its parent's parent, ... up to a root (parent -1)."""
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i]
    return out


def decode_tree(S, z, Q, K, V, W, parents):
    """Outputs [T, d] of T drafted nodes over the state S (m x d), z (m), which is not changed. Each row
    is taken relative to its own largest exponent (the scale cancels)."""
    T, d = Q.shape
    out = np.empty((T, d))
    for i in range(T):
        J = ancestors(parents, i)
        # log features of the query and the visible keys; the state enters through its own logarithm
        uq = W @ Q[i]
        uk = K[J] @ W.T - 0.5 * np.sum(K[J] ** 2, axis=1, keepdims=True) - 0.5 * np.log(W.shape[0])
        with np.errstate(divide="ignore"):
            lz = np.where(z > 0, np.log(z), -np.inf)
        top = max(np.max(uq + lz), np.max(uq[None, :] + uk))
        weights = np.exp(uq[None, :] + uk - top).sum(axis=1)
        share = np.exp(uq + lz - top)
        mean = np.divide(S, z[:, None], out=np.zeros_like(S), where=z[:, None] > 0)
        out[i] = (weights @ V[J] + share @ mean) / (weights.sum() + share.sum())
    return out


def decode_extend(S, z, K, V, W, index=None):
    """The state after adding the tokens ``index`` (in any order, repeats added again; default all)."""
    index = np.arange(len(K)) if index is None else np.asarray(index, dtype=int)
    pk = phi(K[index], W) if len(index) else np.zeros((0, W.shape[0]))
    return S + pk.T @ V[index], z + pk.sum(axis=0)


def verify(parents, tokens, p, q, u, r):
    """The walk of one sequence from node 0: (path, next token). p: [T, V]; q: [T, V], or None for a draft
    of point masses. The next token is -1 where the target's row has no positive sum."""
    p = np.maximum(np.nan_to_num(np.asarray(p, dtype=np.float64), nan=0.0, posinf=np.inf), 0.0)
    cur, path = 0, [0]
    w, Z = p[0].copy(), 1.0
    for c in range(1, len(parents)):
        if parents[c] != cur:
            continue
        x = tokens[c]
        if not 0 <= x < p.shape[1]:
            continue
        qx = 1.0 if q is None else float(q[cur, x])
        if u[c] * (Z * qx) < w[x]:
            cur = c
            path.append(c)
            w, Z = p[c].copy(), 1.0
        elif q is None:
            Z -= w[x]
            w[x] = 0.0
        else:
            w = np.maximum(w - Z * q[cur].astype(np.float64), 0.0)
            Z = w.sum()
    if not (w.sum() > 0 and np.isfinite(w.sum())):
        w = p[cur]
    total = w.sum()
    if not (total > 0 and np.isfinite(total)):
        return path, -1
    run = np.cumsum(w)
    past = np.nonzero((run > r * run[-1]) & (w > 0))[0]
    return path, int(past[0]) if len(past) else int(np.nonzero(w)[0][-1])
