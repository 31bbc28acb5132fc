"""Beam search with a small language model of decayed linear attention, on random weights.

The path a serving program takes: the prompts of all requests in one packed call
(``la_prefill``), every request's states forked to its hypotheses and then, token by token, the
recurrent form for all hypotheses (``la_decode_step``), the choice among beams x vocabulary
(``beam_select``) and the states that follow it (``fp32_state_reorder``). Projections are plain
matrix products.

    python examples/beam_generation.py [--requests 3] [--beams 4] [--tokens 16]
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

D = 128


class Model:
    """Embedding, layers of linear attention with a decay per head, tied output projection."""

    def __init__(self, vocab=501, width=256, layers=2, heads=4, key_heads=2, dtype=torch.float32, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *shape, scale: (torch.randn(*shape, generator=g) * scale).to(device, dtype)
        self.heads, self.key_heads, self.dtype, self.n_layers = heads, key_heads, dtype, layers
        self.embed = rnd(vocab, width, scale=1.0)
        self.layers = [dict(qkv=rnd(width, (2 * key_heads + heads) * D, scale=width ** -0.5),
                            decay=rnd(width, heads, scale=width ** -0.5),
                            out=rnd(heads * D, width, scale=(heads * D) ** -0.5)) for _ in range(layers)]

    def inputs(self, layer, x):
        """q, k, v (rows of one fused projection, as the calls take them) and decays of tokens x [n][width]."""
        K, H = self.key_heads, self.heads
        x = torch.nn.functional.normalize(x.float(), dim=-1).to(x.dtype) * x.shape[-1] ** 0.5
        q, k, v = (y.unflatten(1, (-1, D)) for y in (x @ layer["qkv"]).split([K * D, K * D, H * D], dim=1))
        k.mul_(D ** -0.5)
        return q, k, v, torch.sigmoid((x @ layer["decay"]).float() + 3.0).contiguous()

    def logits(self, x):
        return (x @ self.embed.T) * x.shape[-1] ** -0.5


def generate(model: Model, prompts, beams=4, tokens=16):
    """(tokens [request][beam][tokens], scores [request][beam]) of the best continuations of each prompt (lists of ids)."""
    dev, R, H, L = model.embed.device, len(prompts), model.heads, model.n_layers
    cfg = lq.la_config(H, model.key_heads, model.dtype)
    lens = [len(p) for p in prompts]
    cu = torch.tensor([0] + lens).cumsum(0).to(dev, torch.int32)
    n, longest = sum(lens), max(lens)
    # states of all layers: [layer][request][beam][head]; a prompt's go to its first beam
    S = torch.zeros(L, R, beams, H, D, D, device=dev)
    ws = torch.empty(lq.la_workspace_bytes(cfg, R, n, longest), dtype=torch.uint8, device=dev)
    x = model.embed[torch.tensor([t for p in prompts for t in p], device=dev)]
    last = torch.empty(R, H, D, D, device=dev)
    for i, layer in enumerate(model.layers):
        q, k, v, a = model.inputs(layer, x)
        o = torch.empty(n, H, D, dtype=model.dtype, device=dev)
        lq.la_prefill(cfg, q, k, v, a, o, cu_seqlens=cu, max_len=longest, S_out=last,
                      workspace=ws if ws.numel() else None)
        S[i, :, 0] = last
        x = x + o.flatten(1) @ layer["out"]
    x = x[cu[1:].long() - 1]
    fork = torch.zeros(R, beams, dtype=torch.int32, device=dev)
    lq.fp32_state_reorder(S, fork, outer=L, inner=H)

    logits = model.logits(x)[:, None].expand(R, beams, -1).contiguous()
    scores = torch.full((R, beams), -torch.inf, device=dev)
    scores[:, 0] = 0.0  # the hypotheses are still the same one
    best, parent, token = (torch.empty(R, beams, dtype=t, device=dev) for t in (torch.float32, torch.int32, torch.int32))
    work = torch.empty(lq.beam_workspace_bytes(R, beams, logits.shape[2], beams), dtype=torch.uint8, device=dev)
    out = torch.empty(R, beams, 0, dtype=torch.int64, device=dev)
    o = torch.empty(R * beams, H, D, dtype=model.dtype, device=dev)
    for step in range(tokens):
        lq.beam_select(logits, scores, best, parent, token, work)
        scores.copy_(best)
        out = torch.cat([out.gather(1, parent.long()[..., None].expand_as(out)), token.long()[..., None]], dim=2)
        if step + 1 == tokens:
            break
        lq.fp32_state_reorder(S, parent, outer=L, inner=H)
        x = model.embed[token.long().flatten()]
        for i, layer in enumerate(model.layers):
            q, k, v, a = model.inputs(layer, x)
            lq.la_decode_step(cfg, S[i], q, k, v, a, o)
            x = x + o.flatten(1) @ layer["out"]
        logits = model.logits(x).view(R, beams, -1)
    return out, scores


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=16)
    a = ap.parse_args()
    model = Model(dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 501, (int(n),), generator=g).tolist() for n in torch.randint(1, 400, (a.requests,), generator=g)]
    out, scores = generate(model, prompts, a.beams, a.tokens)
    for r, p in enumerate(prompts):
        print(f"request {r}: {len(p)} prompt tokens")
        for b in range(a.beams):
            print(f"  {scores[r, b].item():8.3f}  {out[r, b].tolist()}")


if __name__ == "__main__":
    main()
