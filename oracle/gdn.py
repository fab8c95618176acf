"""Plain float64 gated delta rule and draft verification on the CPU, for the tests.

gdn_run: per value head, S <- exp(g) S; e = beta (v - S k); S <- S + e k^T;
o = scale S q, token after token; value head h reads query/key head h // (Hv / Hk).
verify_drafts: the accept/reject rule with its comparisons in float32, entry by entry.
Shares no code with the library or with the other oracle.
"""
from __future__ import annotations

import numpy as np


def _lengths(x, eps):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + eps) if eps > 0 else x


def gdn_run(S0, q, k, v, g, beta, scale, eps, every=False, round_state=None):
    """One sequence: S0 [Hv, dv, dk]; q, k [T, Hk, dk]; v [T, Hv, dv]; g, beta [T, Hv].
    Returns (o [T, Hv, dv], S, states after every token or None).  round_state is applied
    to the state after each token (a pool that stores rounded states)."""
    S = np.array(S0, dtype=np.float64)
    share = v.shape[1] // q.shape[1]
    q = np.repeat(_lengths(np.asarray(q, np.float64), eps), share, axis=1) * scale
    k = np.repeat(_lengths(np.asarray(k, np.float64), eps), share, axis=1)
    v, g, beta = (np.asarray(x, np.float64) for x in (v, g, beta))
    o = np.zeros(v.shape)
    kept = []
    for t in range(len(v)):
        S = S * np.exp(g[t])[:, None, None]
        e = beta[t][:, None] * (v[t] - np.einsum("hij,hj->hi", S, k[t]))
        S = S + e[:, :, None] * k[t][:, None, :]
        o[t] = np.einsum("hij,hj->hi", S, q[t])
        if round_state is not None:
            S = round_state(S)
        if every:
            kept.append(S.copy())
    return o, S, (np.stack(kept) if every else None)


def verify_drafts(draft_ids, p, q, uniforms, noise, n_draft=None):
    """Rows of drafts (all arrays float32 / int): (accepted [n], tokens [n, K+1])."""
    n, K = draft_ids.shape
    f32 = np.float32
    accepted = np.zeros(n, np.int32)
    tokens = np.full((n, K + 1), -1, np.int32)
    with np.errstate(all="ignore"):
        for b in range(n):
            drafted = K if n_draft is None else int(n_draft[b])
            m = 0
            while m < drafted:
                x = draft_ids[b, m]
                qx = f32(1.0) if q is None else f32(q[b, m, x])
                if not f32(uniforms[b, m]) * qx < f32(p[b, m, x]):
                    break
                tokens[b, m] = x
                m += 1
            accepted[b] = m
            rest = np.asarray(p[b, m], f32)
            if m < drafted:
                if q is not None:
                    rest = rest - np.asarray(q[b, m], f32)
                else:
                    rest = rest.copy()
                    rest[draft_ids[b, m]] = 0
                if not (rest > 0).any():
                    rest = np.asarray(p[b, m], f32)
            best, at = f32(-1.0), -1
            score = rest / np.asarray(noise[b], f32)
            for x in np.flatnonzero(rest > 0):
                if score[x] > best:
                    best, at = score[x], x
            tokens[b, m] = at
    return accepted, tokens
