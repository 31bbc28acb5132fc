"""Plain 64-bit forms of the generation operators, and the errors their tests allow."""
from __future__ import annotations

import numpy as np

D = 128


def half_step(dtype) -> float:
    """The largest relative error of one rounding to nearest."""
    import torch

    return torch.finfo(dtype).eps / 2


def la_reference(q, k, v, alpha, lens, S0=None):
    """o and last states of S_t = alpha_t S_{t-1} + v_t k_t^T, o_t = S_t q_t, token by token; q, k [T][K][D],
    v [T][H][D], alpha [T][H] as float64 arrays, the sequences one after the other."""
    H, many = v.shape[1], v.shape[1] // k.shape[1]
    o = np.zeros(v.shape)
    S = np.zeros((len(lens), H, D, D)) if S0 is None else np.array(S0, dtype=np.float64)
    t = 0
    with np.errstate(all="ignore"):
        for b, n in enumerate(lens):
            for _ in range(n):
                kk, qq = np.repeat(k[t], many, axis=0), np.repeat(q[t], many, axis=0)
                S[b] = alpha[t][:, None, None] * S[b] + v[t][:, :, None] * kk[:, None, :]
                o[t] = np.einsum("hij,hj->hi", S[b], qq)
                t += 1
    return o, S


def state_bound(longest) -> float:
    """Relative L2 error of an fp32 state, or of an fp32 output, after `longest` tokens: every token rounds the
    sums and every product chain of 128 rounds its partial sums, each by 2^-24 at most and with either sign, so
    they add as a random walk; twice that, and eight roundings for the decays' logarithms and powers."""
    return 2.0 ** -24 * (8 + 2 * np.sqrt(128 + longest))


def output_bound(dtype, longest) -> float:
    """Relative L2 error of o: in 16-bit types the result is rounded once and the chunk's products and the state
    may be rounded once each before they are summed, half a step at most each with either sign: sqrt(3) of
    them, below twice; fp32 sums beneath."""
    import torch

    return state_bound(longest) + (0.0 if dtype == torch.float32 else 2 * half_step(dtype))


def rel(a, b) -> float:
    n = np.linalg.norm(b)
    return float(np.linalg.norm(a - b) / n) if n else float(np.linalg.norm(a - b) != 0)


def beam_reference(logits, scores, n_best):
    """(scores, parent, token) in 64 bits; dead hypotheses (a score or log-sum-exp that is not finite) score -inf."""
    B, K, V = logits.shape
    x = np.asarray(logits, np.float64)
    s = np.full((B, K, V), -np.inf)
    with np.errstate(all="ignore"):
        for b in range(B):
            for k in range(K):
                top = x[b, k].max()
                if not np.isfinite(top) or not np.isfinite(scores[b, k]):
                    continue
                lse = top + np.log(np.exp(x[b, k] - top).sum())
                s[b, k] = float(scores[b, k]) + (x[b, k] - lse)
    flat = s.reshape(B, K * V)
    order = np.argsort(-flat, axis=1, kind="stable")[:, :n_best]
    return np.take_along_axis(flat, order, 1), order // V, order % V


def reorder_reference(planes, parent, outer, inner, counts=None):
    """Planes [N, ...] after the reordering; planes named rec_* move the source's records only."""
    G, K = parent.shape
    out = {}
    for name, x in planes.items():
        old = x.reshape(outer, G, K, inner, *x.shape[1:])
        new = old.copy()
        for o in range(outer):
            for g in range(G):
                if parent[g].min() < 0 or parent[g].max() >= K:
                    continue
                for b in range(K):
                    for i in range(inner):
                        src = parent[g, b]
                        if src == b:
                            continue
                        n = x.shape[1] if x.ndim > 1 else None
                        if name.startswith("rec_"):
                            c = int(counts.reshape(outer, G, K, inner)[o, g, src, i])
                            n = c * (x.shape[1] // counts_window(planes))
                        if n is None:
                            new[o, g, b, i] = old[o, g, src, i]
                        else:
                            new[o, g, b, i, :n] = old[o, g, src, i, :n]
        out[name] = new.reshape(x.shape)
    return out


def counts_window(planes) -> int:
    return planes["rec_k"].shape[1]
