"""The generation operators' measured cases and their plain forms.

Four operators: linear attention with a decay for each head over prompts
(chunked), the same for single tokens on fp32 states (recurrent), the selection
of beam search over beams and vocabulary, and the reordering of head-states
after it (quantized state buffers and fp32 states). Where ``own`` is false the
plain forms below run; where it is true the framework's calls do.
"""
import math
import random

import torch

own = False

D = 128  # key and value channels of a head-state
CHUNK = 64  # tokens per chunk of the plain prompt form
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a chat turn: one short prompt on a small model; latency counts
        dict(name="prompt_short", op="prefill", dtype="bf16", seqs=1, max_len=77, heads=4, key_heads=4, first=False,
             fused=False),
        # an engine's prefill batch: ragged prompts (one of them empty), shared key heads, rows of one fused
        # projection, states carried over from an earlier part of each prompt
        dict(name="prompt_ragged", op="prefill", dtype="bf16", seqs=16, max_len=1500, heads=32, key_heads=8,
             first=True, fused=True),
        # one long document: few head-states, a long axis to split
        dict(name="prompt_long", op="prefill", dtype="bf16", seqs=1, max_len=32768, heads=32, key_heads=32,
             first=False, fused=False),
        # full precision, the type the framework's own decode calls take
        dict(name="prompt_fp32", op="prefill", dtype="f32", seqs=4, max_len=2048, heads=16, key_heads=16, first=True,
             fused=False),
        # one request, one layer, one token
        dict(name="token_one_request", op="step", dtype="bf16", seqs=1, heads=32, key_heads=8),
        # the batch-512 layer of the framework's benchmark: 16384 head-states
        dict(name="token_batch", op="step", dtype="bf16", seqs=512, heads=32, key_heads=32),
        # one interactive request with four hypotheses; latency counts
        dict(name="beams_one_request", op="select", dtype="bf16", batch=1, beams=4, vocab=32000, n_best=8,
             masked=False, begin=False, padded=False),
        # a grammar-constrained batch in full precision, odd vocabulary, rows padded in memory
        dict(name="beams_masked", op="select", dtype="f32", batch=16, beams=5, vocab=50257, n_best=10, masked=True,
             begin=False, padded=True),
        # a serving batch with a large odd vocabulary
        dict(name="beams_batch", op="select", dtype="bf16", batch=64, beams=8, vocab=131071, n_best=16, masked=False,
             begin=False, padded=True),
        # one request with four hypotheses, sixteen layers
        dict(name="reorder_one_request", op="reorder", kind="lq", kda=False, outer=16, groups=1, beams=4, inner=32),
        # 128 requests with four hypotheses each: 16384 quantized head-states of one layer
        dict(name="reorder_batch", op="reorder", kind="lq", kda=False, outer=1, groups=128, beams=4, inner=32),
        # the unquantized baseline's states
        dict(name="reorder_fp32", op="reorder", kind="fp32", kda=False, outer=8, groups=4, beams=8, inner=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "select", "reorder"])
    if op == "prefill":
        heads = rng.choice([1, 2, 4, 6, 8, 12, 16, 24, 32])
        key_heads = rng.choice([h for h in range(1, heads + 1) if heads % h == 0])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        room = (1 << 20) // heads // (2 if dtype == "f32" else 1)  # padded tokens of all sequences
        max_len = _log_int(rng, 1, min(32768, room))
        seqs = _log_int(rng, 1, max(1, min(64, room // max_len)))
        return dict(op=op, dtype=dtype, seqs=seqs, max_len=max_len, heads=heads, key_heads=key_heads,
                    first=rng.random() < 0.5, fused=rng.random() < 0.5)
    if op == "step":
        heads = rng.choice([1, 3, 4, 8, 16, 32])
        key_heads = rng.choice([h for h in range(1, heads + 1) if heads % h == 0])
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), seqs=_log_int(rng, 1, 512), heads=heads,
                    key_heads=key_heads)
    if op == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), batch=_log_int(rng, 1, 512 // beams // 2),
                    beams=beams, vocab=_log_int(rng, 1000, 131071), n_best=beams * rng.choice([1, 2]),
                    masked=rng.random() < 0.3, begin=rng.random() < 0.2, padded=rng.random() < 0.5)
    beams = rng.choice([2, 3, 4, 5, 8, 16])
    inner = rng.choice([1, 4, 16, 32])
    room = 16384 // (beams * inner)
    outer = _log_int(rng, 1, min(32, room))
    return dict(op=op, kind=rng.choice(["lq", "lq", "fp32"]), kda=rng.random() < 0.3, outer=outer,
                groups=_log_int(rng, 1, max(1, room // outer // 2)), beams=beams, inner=inner)


def _lens(case):
    """The sequences' lengths: the first is the longest; of eight or more, the second is empty."""
    rng = random.Random(case["seqs"] * 1000003 + case["max_len"])
    lens = [case["max_len"]] + [_log_int(rng, 1, case["max_len"]) for _ in range(case["seqs"] - 1)]
    if len(lens) >= 8:
        lens[1] = 0
    return lens


def work(case):
    """What a pass cannot do without."""
    if case["op"] == "prefill":
        n, e, lens = case["heads"], SIZES[case["dtype"]], _lens(case)
        T = sum(lens)
        states = (2 if case["first"] else 1) * len(lens) * n * D * D * 4
        return {"bytes": T * (2 * n + 2 * case["key_heads"]) * D * e + 4 * T * n + states, "flops": 4.0 * T * n * D * D}
    if case["op"] == "step":
        n, e, B = case["heads"], SIZES[case["dtype"]], case["seqs"]
        return {"bytes": B * n * D * D * 8 + B * (2 * n + 2 * case["key_heads"]) * D * e + 4 * B * n,
                "flops": 5.0 * B * n * D * D}
    if case["op"] == "select":
        rows = case["batch"] * case["beams"]
        return {"bytes": rows * case["vocab"] * SIZES[case["dtype"]] + 4 * rows + 12 * case["batch"] * case["n_best"],
                "flops": 4.0 * rows * case["vocab"]}
    # the parents are drawn evenly: K - 1 of a group's K beams change on average, and a beam is a source of
    # another one with probability 1 - (1 - 1/K)^(K - 1)
    K = case["beams"]
    moved = (K - 1) + K * (1 - (1 - 1 / K) ** (K - 1))
    if case["kind"] == "fp32":
        per_state = 4 * D * D
    else:  # codes, steps, scales, compensators and half of the window's 16 records
        per_state = D * D + 8 * D + 16 + 4 * 4 * D + 8 * (8 * D + (4 * D if case["kda"] else 4)) + 4
    return {"bytes": case["outer"] * case["groups"] * case["inner"] * moved * per_state, "flops": 0.0}


# ----------------------------------------------------------------------------------------------- inputs
def _normal(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def _decays(gen, tokens, heads):
    """Half-lives from one token to ten thousand, a base for each head and a spread over its tokens."""
    base = torch.rand(heads, generator=gen, device="cuda") * math.log(1e4)
    half = torch.exp(base + 0.5 * torch.randn(tokens, heads, generator=gen, device="cuda"))
    return torch.exp2(-1.0 / half)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"prefill": _prepare_prefill, "step": _prepare_step, "select": _prepare_select,
            "reorder": _prepare_reorder}[case["op"]](case, gen)


def _prepare_prefill(case, gen):
    dt, H, K, lens = DTYPES[case["dtype"]], case["heads"], case["key_heads"], _lens(case)
    T, B = sum(lens), len(lens)
    if case["fused"]:  # one row a token: the key heads' queries, the key heads' keys, the heads' values
        rows = torch.empty(T, (2 * K + H) * D, dtype=dt, device="cuda")
        q, k, v = (x.view(T, -1, D) for x in rows.split([K * D, K * D, H * D], dim=1))
    else:
        q, k, v = (torch.empty(T, n, D, dtype=dt, device="cuda") for n in (K, K, H))
    q.copy_(_normal(gen, T, K, D))
    k.copy_(_normal(gen, T, K, D, scale=D ** -0.5))
    v.copy_(_normal(gen, T, H, D))
    cu = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    s = dict(op="prefill", q=q, k=k, v=v, alpha=_decays(gen, T, H), cu=cu, max_len=max(lens), B=B, H=H, K=K,
             S0=_normal(gen, B, H, D, D, scale=0.3) if case["first"] else None, dtype=dt,
             o=torch.empty(T, H, D, dtype=dt, device="cuda"), S=torch.empty(B, H, D, D, device="cuda"))
    if own:  # what a user's program keeps beside its buffers: the head layout and a workspace
        from quantized_linear_attention_gb300 import lq

        s["cfg"] = lq.la_config(H, K, dt)
        s["workspace"] = torch.empty(lq.la_workspace_bytes(s["cfg"], B, T, max(lens)), dtype=torch.uint8,
                                     device="cuda")
    return s


def _prepare_step(case, gen):
    dt, H, K, B = DTYPES[case["dtype"]], case["heads"], case["key_heads"], case["seqs"]
    s = dict(op="step", S=_normal(gen, B, H, D, D, scale=0.3), q=_normal(gen, B, K, D, dtype=dt),
             k=_normal(gen, B, K, D, scale=D ** -0.5, dtype=dt), v=_normal(gen, B, H, D, dtype=dt),
             alpha=_decays(gen, B, H), o=torch.empty(B, H, D, dtype=dt, device="cuda"), H=H, K=K)
    if own:
        from quantized_linear_attention_gb300 import lq

        s["cfg"] = lq.la_config(H, K, dt)
    return s


def _prepare_select(case, gen):
    B, K, V, M = case["batch"], case["beams"], case["vocab"], case["n_best"]
    wide = -(-V // 64) * 64 if case["padded"] else V
    full = torch.empty(B, K, wide, dtype=DTYPES[case["dtype"]], device="cuda")
    full.copy_(_normal(gen, B, K, wide, scale=2.5))
    logits = full[:, :, :V]
    if case["masked"]:  # a third of the vocabulary is not allowed next
        logits[torch.rand(B, K, V, generator=gen, device="cuda") < 1 / 3] = -math.inf
    scores = -20.0 * torch.rand(B, K, generator=gen, device="cuda").sort(dim=1).values
    if case["begin"]:  # the first selection: only beam 0 is alive
        scores[:, 1:] = -math.inf
    s = dict(op="select", logits=logits, scores=scores, M=M, out_scores=torch.empty(B, M, device="cuda"),
             parent=torch.empty(B, M, dtype=torch.int32, device="cuda"),
             token=torch.empty(B, M, dtype=torch.int32, device="cuda"))
    if own:
        from quantized_linear_attention_gb300 import lq

        s["workspace"] = torch.empty(lq.beam_workspace_bytes(B, K, V, M), dtype=torch.uint8, device="cuda")
    return s


def _prepare_reorder(case, gen):
    O, G, K, I = case["outer"], case["groups"], case["beams"], case["inner"]
    N, W, C = O * G * K * I, 16, 4
    s = dict(op="reorder", outer=O, inner=I, N=N,
             parent=torch.randint(0, K, (G, K), generator=gen, device="cuda", dtype=torch.int32))
    if case["kind"] == "fp32":
        s["planes"] = {"S": _normal(gen, N, D, D)}
        return s
    # a request's hypotheses are at the same token: one record count for each group
    counts = torch.randint(0, W + 1, (1, G, 1, 1), generator=gen, device="cuda", dtype=torch.int32)
    planes = {
        "counts": counts.expand(O, G, K, I).reshape(N).contiguous(),
        "codes": torch.randint(-127, 128, (N, D, D), generator=gen, device="cuda", dtype=torch.int8),
        "sigma": _normal(gen, N, D).abs(),
        "lambda": _normal(gen, N, D).abs(),
        "comp_id": torch.randint(0, 2 * D, (N, C), generator=gen, device="cuda", dtype=torch.int32),
        "comp_line": _normal(gen, N, C, D),
        "rec_k": _normal(gen, N, W, D),
        "rec_u": _normal(gen, N, W, D),
        "rec_alpha": torch.rand(N, W * D if case["kda"] else W, generator=gen, device="cuda"),
    }
    if own:  # the same planes in a state buffer, the handle that the framework's calls take
        from quantized_linear_attention_gb300 import lq

        s["cfg"] = lq.config(window=W, n_comp=C, kda=case["kda"])
        s["state"] = lq.alloc_state(s["cfg"], N)
        lq.state_init(s["cfg"], s["state"], N, None)
        views = lq.state_views(s["cfg"], s["state"], N)
        for name in planes:
            views[name].copy_(planes[name])
        planes = {name: views[name] for name in planes}
    s["planes"] = planes
    return s


# ------------------------------------------------------------------------------------------------- runs
def run(s):
    if own:
        from quantized_linear_attention_gb300 import lq

        if s["op"] == "prefill":
            lq.la_prefill(s["cfg"], s["q"], s["k"], s["v"], s["alpha"], s["o"], cu_seqlens=s["cu"],
                          max_len=s["max_len"], S0=s["S0"], S_out=s["S"], workspace=s["workspace"])
            return {"o": s["o"], "S": s["S"]}
        if s["op"] == "step":
            lq.la_decode_step(s["cfg"], s["S"], s["q"], s["k"], s["v"], s["alpha"], s["o"])
            return {"o": s["o"], "S": s["S"]}
        if s["op"] == "select":
            lq.beam_select(s["logits"], s["scores"], s["out_scores"], s["parent"], s["token"], s["workspace"])
            return {"scores": s["out_scores"], "parent": s["parent"], "token": s["token"]}
        if "S" in s["planes"]:
            lq.fp32_state_reorder(s["planes"]["S"], s["parent"], outer=s["outer"], inner=s["inner"])
        else:
            lq.state_reorder(s["cfg"], s["state"], s["N"], s["parent"], outer=s["outer"], inner=s["inner"])
        return s["planes"]
    return {"prefill": _plain_prefill, "step": _plain_step, "select": _plain_select,
            "reorder": _plain_reorder}[s["op"]](s)


def _plain_prefill(s):
    """Chunks of 64 tokens of each sequence, padded to the longest; decays as differences of 64-bit sums of logarithms."""
    B, H, cu = s["B"], s["H"], s["cu"].long()
    N = max(1, -(-s["max_len"] // CHUNK))
    at = cu[:-1, None] + torch.arange(N * CHUNK, device="cuda")
    there = at < cu[1:, None]
    at = torch.where(there, at, 0)

    def rows(x, heads, fill):  # [T, heads, ...] -> [B, H, N, CHUNK, ...], 32 bits
        x = torch.where(there.view(B, -1, *[1] * (x.dim() - 1)), x[at], fill).to(torch.float32)
        x = x.repeat_interleave(H // heads, dim=2).transpose(1, 2)
        return x.reshape(B, H, N, CHUNK, *x.shape[3:])

    q, k, v = rows(s["q"], s["K"], 0), rows(s["k"], s["K"], 0), rows(s["v"], H, 0)
    g = rows(s["alpha"], H, 1).double().log2().view(B, H, -1).cumsum(-1).view(B, H, N, CHUNK)
    ends = torch.cat([torch.zeros(B, H, 1, device="cuda", dtype=torch.float64), g[..., -1]], dim=2)  # before chunk n

    def decay(x):
        return torch.exp2(x).to(torch.float32)

    past = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    inside = decay(torch.where(past, g[..., :, None] - g[..., None, :], -math.inf))
    o = ((q @ k.transpose(-1, -2)) * inside) @ v
    added = (v * decay(g[..., -1:] - g).unsqueeze(-1)).transpose(-1, -2) @ k  # what each chunk adds to the state
    past = torch.ones(N + 1, N, dtype=torch.bool, device="cuda").tril(-1)
    between = decay(torch.where(past, ends[..., :, None] - ends[..., None, 1:], -math.inf))
    S = (between @ added.view(B, H, N, D * D)).view(B, H, N + 1, D, D)
    if s["S0"] is not None:
        S = S + decay(ends)[..., None, None] * s["S0"].unsqueeze(2)
    o = o + decay(g - ends[..., :-1, None]).unsqueeze(-1) * (q @ S[:, :, :-1].transpose(-1, -2))
    o = o.reshape(B, H, N * CHUNK, D).transpose(1, 2)[there]
    return {"o": o.to(s["dtype"]), "S": S[:, :, -1].contiguous()}


def _plain_step(s):
    many = s["H"] // s["K"]
    q, k = (s[n].float().repeat_interleave(many, dim=1) for n in ("q", "k"))
    s["S"].mul_(s["alpha"][..., None, None]).add_(s["v"].float()[..., :, None] * k[..., None, :])
    o = (s["S"] @ q[..., :, None]).squeeze(-1)
    return {"o": o.to(s["o"].dtype), "S": s["S"]}


def _plain_select(s):
    """64 bits: the order of nearly equal candidates of different beams hangs on their log-sum-exp."""
    x = s["logits"].double()
    B, K, V = x.shape
    top = x.amax(-1, keepdim=True)
    lse = top + (x - top).exp().sum(-1, keepdim=True).log()
    scores = s["scores"].double()[..., None] + (x - lse)
    alive = lse.isfinite() & s["scores"].double()[..., None].isfinite()
    scores = torch.where(alive, scores, -math.inf).view(B, K * V)
    best, at = (t[:, :s["M"]] for t in torch.sort(scores, dim=1, descending=True, stable=True))
    return {"scores": best.float(), "parent": (at // V).int(), "token": (at % V).int()}


def _plain_reorder(s):
    G, K = s["parent"].shape
    O, I, planes = s["outer"], s["inner"], s["planes"]
    group = torch.arange(O * G, device="cuda").view(O, G, 1, 1)
    src = ((group * K + s["parent"].view(1, G, K, 1)) * I + torch.arange(I, device="cuda")).view(-1)
    if "counts" in planes:
        n = planes["counts"][src]
        live = torch.arange(planes["rec_k"].shape[1], device="cuda") < n[:, None]  # the source's records
    for name, x in planes.items():
        new = x[src]
        if name.startswith("rec_"):
            W = live.shape[1]
            new = torch.where(live[..., None], new.view(len(new), W, -1), x.reshape(len(new), W, -1)).view(x.shape)
        x.copy_(new)
    return planes


# ------------------------------------------------------------------------------------------ definitions
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefill":
        return _exact_prefill(s, _lens(case))
    if case["op"] == "step":
        S = s["S"].double()
        B, H = S.shape[:2]
        o = torch.empty(B, H, D, dtype=torch.float64, device="cuda")
        for h in range(H):
            kh = h // (H // s["K"])
            S[:, h] = s["alpha"][:, h, None, None].double() * S[:, h] + torch.einsum(
                "bi,bj->bij", s["v"][:, h].double(), s["k"][:, kh].double())
            o[:, h] = torch.einsum("bij,bj->bi", S[:, h], s["q"][:, kh].double())
        return {"o": o, "S": S}
    if case["op"] == "select":
        B, K, V = s["logits"].shape
        best = torch.empty(B, s["M"], dtype=torch.float64, device="cuda")
        for b in range(B):
            logp = s["logits"][b].double()
            logp = logp - torch.logsumexp(logp, dim=1, keepdim=True) + s["scores"][b].double()[:, None]
            best[b] = torch.topk(logp.reshape(-1), s["M"]).values
        return {"scores": best, "parent": None, "token": None}
    O, I, (G, K) = s["outer"], s["inner"], s["parent"].shape
    parent = s["parent"].tolist()
    out = {}
    for name, x in s["planes"].items():
        if not x.is_floating_point():
            out[name] = None
            continue
        old = x.view(O, G, K, I, *x.shape[1:])
        new = old.clone()
        for g in range(G):
            n = int(s["planes"]["counts"].view(O, G, K, I)[0, g, 0, 0]) if "counts" in s["planes"] else 0
            rows = slice(0, n * (x.shape[1] // 16)) if name.startswith("rec_") else slice(None)
            for b in range(K):
                new[:, g, b, :, rows] = old[:, g, parent[g][b], :, rows]
        out[name] = new.view(x.shape) if x.numel() > 1 << 28 else new.view(x.shape).double()
    return out


def _exact_prefill(s, lens):
    """Token by token in 64 bits, the sequences side by side."""
    B, H, many = s["B"], s["H"], s["H"] // s["K"]
    begin = [sum(lens[:i]) for i in range(B)]
    S = torch.zeros(B, H, D, D, dtype=torch.float64, device="cuda") if s["S0"] is None else s["S0"].double()
    o = torch.empty(sum(lens), H, D, dtype=torch.float64, device="cuda")
    order = sorted(range(B), key=lambda i: -lens[i])  # those still running are always the first ones
    S = S[order].contiguous()
    first = torch.tensor([begin[i] for i in order], device="cuda")
    alpha = s["alpha"].double()
    running = B
    for t in range(max(lens)):
        while lens[order[running - 1]] <= t:
            running -= 1
        at = first[:running] + t
        k = s["k"][at].double().repeat_interleave(many, dim=1)
        q = s["q"][at].double().repeat_interleave(many, dim=1)
        live = S[:running]
        live.mul_(alpha[at][..., None, None]).addcmul_(s["v"][at].double()[..., :, None], k[..., None, :])
        o[at] = (live * q[..., None, :]).sum(-1)
    back = torch.empty(B, dtype=torch.long, device="cuda")
    back[torch.tensor(order, device="cuda")] = torch.arange(B, device="cuda")
    return {"o": o, "S": S[back]}
