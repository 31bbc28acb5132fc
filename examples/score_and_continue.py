"""Scoring prompts and going on from them with a small state space language model, on random weights.

The path a serving program takes: the prompts of all requests in one packed call per operator (``conv_prefill``,
``ssm_prefill``), the log probability of every prompt token with the entropy before it and its alternatives
(``token_logprobs``), then token by token the recurrent forms (``conv_decode_step``, ``ssm_decode_step``), each time
taking the most likely token. Projections are plain matrix products.

    python examples/score_and_continue.py [--requests 3] [--tokens 16]
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

from quantized_linear_attention_gb300 import lq


class Model:
    """Embedding, layers of convolution and selective scan with a gate, tied output projection."""

    def __init__(self, vocab=501, width=128, layers=2, n_state=16, taps=4, dtype=torch.float32, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *shape, scale, to=dtype: (torch.randn(*shape, generator=g) * scale).to(device, to)
        inner, rank, f = 2 * width, max(1, width // 16), torch.float32
        self.vocab, self.inner, self.rank, self.n_state, self.taps, self.dtype = vocab, inner, rank, n_state, taps, dtype
        self.embed = rnd(vocab, width, scale=1.0)
        step = torch.exp(torch.linspace(-6.9, -2.3, inner))
        self.layers = [dict(xz=rnd(width, 2 * inner, scale=width ** -0.5), conv=rnd(inner, taps, scale=taps ** -0.5, to=f),
                            conv_bias=rnd(inner, scale=0.1, to=f), sel=rnd(inner, rank + 2 * n_state, scale=inner ** -0.5),
                            dt=rnd(rank, inner, scale=rank ** -0.5), dt_bias=torch.log(torch.expm1(step)).to(device),
                            A=(-torch.arange(1.0, n_state + 1).expand(inner, n_state)).contiguous().to(device),
                            D=torch.ones(inner, device=device), out=rnd(inner, width, scale=inner ** -0.5))
                       for _ in range(layers)]
        self.conv_cfg = lq.conv_config(inner, taps, dtype)
        self.ssm_cfg = lq.ssm_config(inner, n_state, 1, dtype)

    def states(self, n_seqs):
        """Convolution inputs and scan states of every layer, zero."""
        L, dev = len(self.layers), self.embed.device
        return (torch.zeros(L, n_seqs, self.taps - 1, self.inner, dtype=self.dtype, device=dev),
                torch.zeros(L, n_seqs, self.inner, self.n_state, device=dev))

    def forward(self, tokens, states, cu=None, longest=0, workspace=None):
        """Logits after each token: packed prompts where `cu` is given, else one token for each sequence. States move on."""
        x = self.embed[tokens]
        prompts = cu is not None
        for i, w in enumerate(self.layers):
            conv, ssm = states[0][i], states[1][i]
            h = torch.nn.functional.normalize(x.float(), dim=-1).to(x.dtype) * x.shape[-1] ** 0.5
            u, z = (h @ w["xz"]).chunk(2, dim=1)
            v, y = torch.empty_like(u, memory_format=torch.contiguous_format), torch.empty_like(u, memory_format=torch.contiguous_format)
            if prompts:
                lq.conv_prefill(self.conv_cfg, u, w["conv"], v, bias=w["conv_bias"], cu_seqlens=cu, max_len=longest, S0=conv, S_out=conv)
            else:
                lq.conv_decode_step(self.conv_cfg, conv, u, w["conv"], v, bias=w["conv_bias"])
            r, B, C = (v @ w["sel"]).split([self.rank, self.n_state, self.n_state], dim=1)
            dt, B, C = r @ w["dt"], B.unsqueeze(1), C.unsqueeze(1)
            if prompts:
                lq.ssm_prefill(self.ssm_cfg, v, dt, w["A"], B, C, y, D=w["D"], z=z, dt_bias=w["dt_bias"], cu_seqlens=cu,
                               max_len=longest, S0=ssm, S_out=ssm, workspace=workspace)
            else:
                lq.ssm_decode_step(self.ssm_cfg, ssm, v, dt, w["A"], B, C, y, D=w["D"], z=z, dt_bias=w["dt_bias"])
            x = x + y @ w["out"]
        return (x @ self.embed.T) * x.shape[-1] ** -0.5


def score_and_continue(model: Model, prompts, tokens=16, alternatives=3):
    """For each prompt (a list of ids): the log probabilities of its tokens after the first, the entropies before them, the
    likeliest alternatives, and `tokens` more tokens with their log probabilities."""
    dev, R = model.embed.device, len(prompts)
    lens = [len(p) for p in prompts]
    cu = torch.tensor([0] + lens).cumsum(0).to(dev, torch.int32)
    n, longest = sum(lens), max(lens)
    ids = torch.tensor([t for p in prompts for t in p], device=dev)
    states = model.states(R)
    ws = torch.empty(lq.ssm_workspace_bytes(model.ssm_cfg, R, n, longest), dtype=torch.uint8, device=dev)
    logits = model.forward(ids, states, cu, longest, ws if ws.numel() else None)
    target = torch.full((n,), -1, dtype=torch.int32, device=dev)  # nothing follows a prompt's last token
    target[:-1] = ids[1:]
    target[cu[1:].long() - 1] = -1
    logprob, entropy = torch.empty(n, device=dev), torch.empty(n, device=dev)
    top, top_token = torch.empty(n, alternatives, device=dev), torch.empty(n, alternatives, dtype=torch.int32, device=dev)
    lq.token_logprobs(logits, target, logprob, entropy=entropy, top_logprob=top, top_token=top_token)
    last = cu[1:].long() - 1
    token, out, out_logprob = top_token[last, 0], [], []
    best, best_token = top[last, :1], None
    for step in range(tokens):
        out.append(token)
        out_logprob.append(best[:, 0])
        if step + 1 == tokens:
            break
        logits = model.forward(token.long(), states)
        best, best_token = torch.empty(R, 1, device=dev), torch.empty(R, 1, dtype=torch.int32, device=dev)
        lq.token_logprobs(logits, top_logprob=best, top_token=best_token)
        token = best_token[:, 0]
    return dict(logprob=logprob.split(lens), entropy=entropy.split(lens), top=top.split(lens), top_token=top_token.split(lens),
                tokens=torch.stack(out, 1), tokens_logprob=torch.stack(out_logprob, 1))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--tokens", type=int, default=16)
    a = ap.parse_args()
    model = Model(dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 501, (int(n),), generator=g).tolist() for n in torch.randint(1, 400, (a.requests,), generator=g)]
    r = score_and_continue(model, prompts, a.tokens)
    for i, p in enumerate(prompts):
        print(f"request {i}: {len(p)} prompt tokens, log probability {r['logprob'][i].sum().item():.2f}, "
              f"mean entropy {r['entropy'][i].mean().item():.3f}")
        print(f"  {r['tokens'][i].tolist()}  ({r['tokens_logprob'][i].sum().item():.3f})")


if __name__ == "__main__":
    main()
