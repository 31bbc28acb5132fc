"""Convolution, scan and log probabilities together, as examples/score_and_continue.py uses them, against the same model
in 64 bits on the host."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from quantized_linear_attention_gb300 import lq

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


class Plain:
    """The model one token at a time in 64 bits."""

    def __init__(self, m):
        f = lambda t: t.double().cpu().numpy()
        self.E, self.layers = f(m.embed), [{k: f(v) for k, v in w.items()} for w in m.layers]
        self.rank, self.N, L = m.rank, m.n_state, len(m.layers)
        self.line = np.zeros((L, m.taps, m.inner))
        self.h = np.zeros((L, m.inner, m.n_state))

    def feed(self, t):
        x = self.E[t]
        for i, w in enumerate(self.layers):
            u, z = np.split(x / np.linalg.norm(x) * len(x) ** 0.5 @ w["xz"], 2)
            self.line[i] = np.concatenate([self.line[i][1:], u[None]])
            s = (self.line[i] * w["conv"].T).sum(0) + w["conv_bias"]
            v = s / (1 + np.exp(-s))
            r, B, C = np.split(v @ w["sel"], [self.rank, self.rank + self.N])
            d = np.logaddexp(r @ w["dt"] + w["dt_bias"], 0)
            self.h[i] = np.exp(d[:, None] * w["A"]) * self.h[i] + (d * v)[:, None] * B
            x = x + ((self.h[i] @ C + w["D"] * v) * z / (1 + np.exp(-z))) @ w["out"]
        logits = self.E @ x * len(x) ** -0.5
        return logits - logits.max() - np.log(np.exp(logits - logits.max()).sum())


def test_scores_and_tokens_match_the_plain_model():
    """fp32 tokens: the two differ by fp32's rounding alone (through fp32 matrix products of up to 256 terms and two
    layers), far less than the gaps between candidates of this seed."""
    from score_and_continue import Model, score_and_continue

    lq.load()
    torch.backends.cuda.matmul.allow_tf32 = False
    model = Model(vocab=97, width=64, layers=2, dtype=torch.float32, seed=5)
    prompts = [[5], list(range(40, 70)), [7, 7, 7, 80] * 150, [1, 2]]
    r = score_and_continue(model, prompts, tokens=5, alternatives=4)
    for i, p in enumerate(prompts):
        plain = Plain(model)
        for j, t in enumerate(p):
            logp = plain.feed(t)
            want = logp[p[j + 1]] if j + 1 < len(p) else 0.0
            assert abs(r["logprob"][i][j].item() - want) <= 1e-3, (i, j)
            assert abs(r["entropy"][i][j].item() + (np.exp(logp) * logp).sum()) <= 1e-3
            assert np.allclose(r["top"][i][j].cpu().numpy(), np.sort(logp)[::-1][:4], atol=1e-3)
        for j in range(5):
            t = int(np.argmax(logp))
            assert r["tokens"][i, j].item() == t, (i, j)
            assert abs(r["tokens_logprob"][i, j].item() - logp[t]) <= 1e-3
            logp = plain.feed(t)


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "score_and_continue.py"), "--requests", "2",
                        "--tokens", "4"], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("request") == 2
