"""Plain 64-bit forms of the state space layer's operators and of token log probabilities, and the errors their tests allow."""
from __future__ import annotations

import numpy as np


def half_step(dtype) -> float:
    """The largest relative error of one rounding to nearest."""
    import torch

    return torch.finfo(dtype).eps / 2


def smallest(dtype) -> float:
    """Half of the smallest subnormal step: the largest error of a rounding next to zero."""
    import torch

    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def silu(x):
    with np.errstate(all="ignore"):
        return x / (1 + np.exp(-x))


def conv_reference(x, w, bias, lens, S0, act):
    """y, last inputs and the sums of the terms' magnitudes; x [T][C], w [C][W], S0 [B][W-1][C] or None."""
    W, C, B = w.shape[1], w.shape[0], len(lens)
    y, mag, S = np.zeros(x.shape), np.zeros(x.shape), np.zeros((B, W - 1, C))
    t = 0
    for b, n in enumerate(lens):
        line = np.concatenate([np.zeros((W - 1, C)) if S0 is None else S0[b], x[t:t + n]])
        for i in range(n):
            y[t + i] = (line[i:i + W] * w.T).sum(0) + (0 if bias is None else bias)
            mag[t + i] = (np.abs(line[i:i + W]) * np.abs(w.T)).sum(0) + (0 if bias is None else np.abs(bias))
        S[b] = line[n:]
        t += n
    return (silu(y) if act else y), S, mag


def conv_bound(y, mag, dtype):
    """One rounding of y; beneath it at most five roundings of the sum, 2^-24 of its terms' magnitudes each, times
    silu's steepest slope 1.1, and silu's own 2^-21: 13.5 x 2^-24, below 2^-20."""
    return half_step(dtype) * np.abs(y) + smallest(dtype) + 2.0 ** -20 * mag


def softplus(v):
    return np.logaddexp(v, 0.0)


def ssm_reference(x, dt, A, B, C, lens, D=None, z=None, bias=None, S0=None, plus=True):
    """(y, last states) of the recurrence token by token, and a bound on an fp32 evaluation's error of each (without y's
    final rounding). x, dt, z [T][ch], A [ch][N], B, C [T][G][N], S0 [n][ch][N].

    The bound goes along with the recurrence. With d exact to 2^-20 (its sum's rounding and a softplus good to 2^-21), a
    decay exp(d A) is off by 2^-22 of itself for its own evaluation and by |d A| (2^-20 + 2^-22) for its exponent (three
    roundings and d's error); d x B by 2^-20 + 2^-23; the fma by 2^-24 of the terms' magnitudes, which M sums. Where a
    sequence is split, the decay over a segment is one such exponential of a sum of d, whose error stays below what its
    tokens' decays are allowed one by one. y adds a rounding per state, three for D x and the gate, and 2^-20 for silu."""
    T, ch = x.shape
    G, many = B.shape[1], ch // B.shape[1]
    N, n_seqs = A.shape[1], len(lens)
    S = np.zeros((n_seqs, ch, N)) if S0 is None else np.array(S0, np.float64)
    E, M = np.zeros_like(S), np.abs(S)
    y, Ey = np.zeros(x.shape), np.zeros(x.shape)
    u = 2.0 ** -24
    t = 0
    with np.errstate(all="ignore"):
        for b, n in enumerate(lens):
            for _ in range(n):
                d = dt[t] + (0 if bias is None else bias)
                d = softplus(d) if plus else d
                e = d[:, None] * A
                a = np.exp(e)
                add = (d * x[t])[:, None] * np.repeat(B[t], many, axis=0)
                Cc = np.repeat(C[t], many, axis=0)
                E[b] = a * E[b] + a * M[b] * (4 * u + 20 * u * np.abs(e)) + np.abs(add) * 18 * u
                S[b] = a * S[b] + add
                M[b] = a * M[b] + np.abs(add)
                E[b] += 2 * u * M[b] + 2.0 ** -140
                o, m = (Cc * S[b]).sum(1), (np.abs(Cc) * M[b]).sum(1)
                err = (np.abs(Cc) * E[b]).sum(1) + (N + 2) * u * m
                if D is not None:
                    o, m = o + D * x[t], m + np.abs(D * x[t])
                    err += 2 * u * m
                if z is not None:
                    g = silu(z[t])
                    o, err = o * g, np.abs(g) * (err + 18 * u * m)
                y[t], Ey[t] = o, err
                t += 1
    return y, S, Ey, E


def logprob_reference(x, tokens, n_top):
    """(logprob, entropy, top logprob, top token) of rows x [R][V] in 64 bits."""
    R, V = x.shape
    x = np.asarray(x, np.float64)
    lp, H = np.full(R, np.nan), np.full(R, np.nan)
    tl, ti = np.full((R, n_top), np.nan), np.full((R, n_top), -1)
    for r in range(R):
        top = x[r].max()
        if np.isfinite(top):
            p = np.exp(x[r] - top)
            ls = np.log(p.sum())
            with np.errstate(all="ignore"):
                H[r] = ls - np.where(p > 0, p * (x[r] - top), 0).sum() / p.sum()
            order = np.argsort(-x[r], kind="stable")[:n_top]
            ti[r], tl[r] = order, x[r][order] - top - ls
            if 0 <= tokens[r] < V:
                lp[r] = x[r][tokens[r]] - top - ls
        if tokens[r] < 0:
            lp[r] = 0.0
    return lp, H, tl, ti


def logprob_bounds(V, lp, H):
    """Of a log probability and of an entropy. A term of the sum is off by 2^-22 for its exponential and by 2^-23 of its
    exponent, which weighs in by at most log V + 1 on average (terms e^-u u are small where u is large); a thread adds at
    most V / 128 terms and 64 more join them, 2^-24 each. A log probability adds two roundings of its own size; the
    entropy is a weighted mean of exponents of the same relative error."""
    u = 2.0 ** -24
    s = u * (4 + 2 * (np.log(V) + 1) + 64 + V / 128)
    return s + 3 * u * (np.abs(lp) + np.log(V)), s * (3 + 2 * np.log(V)) + 3 * u * np.abs(H)
