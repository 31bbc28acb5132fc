"""Prompts, single tokens, beam selection and reordering together, as examples/beam_generation.py uses them,
against the same search in 64 bits on the host."""
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
D = 128


def plain_search(model, prompt, beams, tokens):
    """Every hypothesis with its own states, one token at a time."""
    f = lambda t: t.double().cpu().numpy()
    layers = [{n: f(w) for n, w in layer.items()} for layer in model.layers]
    E, H, K = f(model.embed), model.heads, model.key_heads

    def feed(S, t):
        x = E[t]
        for i, layer in enumerate(layers):
            y = x / np.linalg.norm(x) * len(x) ** 0.5
            q, k, v = np.split((y @ layer["qkv"]).reshape(-1, D), [K, 2 * K])
            k = k * D ** -0.5
            a = 1 / (1 + np.exp(-(y @ layer["decay"] + 3.0)))
            kk, qq = np.repeat(k, H // K, axis=0), np.repeat(q, H // K, axis=0)
            S[i] = a[:, None, None] * S[i] + v[:, :, None] * kk[:, None, :]
            x = x + np.einsum("hij,hj->hi", S[i], qq).reshape(-1) @ layer["out"]
        z = E @ x * len(x) ** -0.5
        return z - z.max() - np.log(np.exp(z - z.max()).sum())

    S = np.zeros((len(layers), H, D, D))
    for t in prompt:
        logp = feed(S, t)
    live = [(0.0, [], S, logp)]
    for _ in range(tokens):
        cand = sorted(((s + lp[t], -b, -t) for b, (s, _, _, lp) in enumerate(live) for t in range(len(lp))), reverse=True)
        new = []
        for s, b, t in cand[:beams]:
            S = live[-b][2].copy()
            new.append((s, live[-b][1] + [-t], S, feed(S, -t)))
        live = new
    return [(s, toks) for s, toks, _, _ in live]


def test_search_matches_the_plain_one():
    """fp32 tokens: the two differ by fp32's rounding alone, far less than the gaps between candidates of this seed."""
    from beam_generation import Model, generate

    lq.load()
    model = Model(vocab=89, width=64, layers=2, heads=4, key_heads=2, dtype=torch.float32, seed=3)
    prompts = [[5], list(range(40, 70)), [7, 7, 7, 80] * 40]
    out, scores = generate(model, prompts, beams=3, tokens=6)
    for r, p in enumerate(prompts):
        for b, (s, toks) in enumerate(plain_search(model, p, 3, 6)):
            assert out[r, b].tolist() == toks, (r, b)
            assert abs(scores[r, b].item() - s) <= 1e-3


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "beam_generation.py"), "--requests", "2",
                        "--beams", "3", "--tokens", "4"], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("request") == 2
