"""Measured cases of the operators around a selective state space layer, with their plain forms.

Five operators: a layer's short causal convolution over packed prompts and for single tokens, the selective state
space scan over packed prompts and for single tokens, and the log probabilities of given tokens with entropy and top
alternatives. Where ``own`` is false the plain forms below run; where it is true the framework's calls do.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a chat turn: one short prompt on a small layer in full precision; latency counts
        dict(name="conv_short", op="conv", dtype="f32", seqs=1, max_len=77, channels=2048, width=4, silu=True,
             bias=True, first=False, fused=False),
        # an engine's prefill batch: ragged prompts (one of them empty) that go on from an earlier part, queries, keys
        # and values of a layer side by side in the rows of one fused projection
        dict(name="conv_ragged", op="conv", dtype="bf16", seqs=16, max_len=1500, channels=8192, width=4, silu=True,
             bias=False, first=True, fused=True),
        # one request, one layer, one token
        dict(name="conv_token_one", op="conv_step", dtype="bf16", seqs=1, channels=8192, width=4, silu=True, bias=True),
        # a batch of 512 requests
        dict(name="conv_token_batch", op="conv_step", dtype="bf16", seqs=512, channels=8192, width=4, silu=True,
             bias=True),
        # a chat turn: one short prompt; latency counts
        dict(name="scan_short", op="scan", dtype="bf16", seqs=1, max_len=77, channels=2048, n_state=16, groups=1,
             softplus=True, gate=True, first=False, fused=False),
        # an engine's prefill batch: ragged prompts (one of them empty) that go on from an earlier part; x and z are
        # the halves of one projection's rows, dt's, B's and C's sources the parts of another's
        dict(name="scan_ragged", op="scan", dtype="bf16", seqs=16, max_len=1500, channels=4096, n_state=16, groups=1,
             softplus=True, gate=True, first=True, fused=True),
        # one long document: few channels beside each other, a long axis to split
        dict(name="scan_long", op="scan", dtype="bf16", seqs=1, max_len=16384, channels=4096, n_state=16, groups=1,
             softplus=True, gate=True, first=False, fused=False),
        # one request, one layer, one token
        dict(name="token_one", op="step", dtype="bf16", seqs=1, channels=4096, n_state=16, groups=1, softplus=True,
             gate=True),
        # a batch of 512 requests
        dict(name="token_batch", op="step", dtype="bf16", seqs=512, channels=4096, n_state=16, groups=1, softplus=True,
             gate=True),
        # the next token's alternatives for one interactive request; latency counts
        dict(name="logprob_one", op="logprob", dtype="bf16", rows=1, vocab=32000, top=5, masked=False, padded=False),
        # a decoding batch's sampled tokens with twenty alternatives, full precision, a large odd vocabulary, a grammar
        dict(name="logprob_batch", op="logprob", dtype="f32", rows=128, vocab=131071, top=20, masked=True, padded=True),
        # a prompt's own tokens scored, an odd vocabulary without padding
        dict(name="logprob_prompt", op="logprob", dtype="bf16", rows=4096, vocab=50257, top=1, masked=False,
             padded=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _channels(rng, lo, hi):
    """Mostly whole multiples of 64, some odd."""
    c = _log_int(rng, lo, hi)
    return c if rng.random() < 0.3 else max(64, c // 64 * 64)


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan", "step", "logprob", "logprob"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "conv":
        channels = _channels(rng, 64, 12288)
        room = (1 << 26) // channels  # padded tokens of all sequences
        max_len = _log_int(rng, 1, min(32768, room))
        return dict(op=op, dtype=dtype, seqs=_log_int(rng, 1, max(1, min(64, room // max_len))), max_len=max_len,
                    channels=channels, width=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.8,
                    bias=rng.random() < 0.5, first=rng.random() < 0.5, fused=rng.random() < 0.5)
    if op == "conv_step":
        return dict(op=op, dtype=dtype, seqs=_log_int(rng, 1, 512), channels=_channels(rng, 64, 12288),
                    width=rng.choice([2, 3, 4, 4]), silu=rng.random() < 0.8, bias=rng.random() < 0.5)
    if op in ("scan", "step"):
        groups = rng.choice([1, 1, 1, 2, 8])
        channels = max(1, _channels(rng, 64, 8192) // groups) * groups
        n_state = rng.choice([8, 16, 16, 16, 32, 64, 12])
        if op == "step":
            return dict(op=op, dtype=dtype, seqs=_log_int(rng, 1, min(512, (1 << 25) // (channels * n_state))),
                        channels=channels, n_state=n_state, groups=groups, softplus=rng.random() < 0.8,
                        gate=rng.random() < 0.7)
        room = (1 << 29) // (channels * n_state)
        max_len = _log_int(rng, 1, min(16384, room))
        return dict(op=op, dtype=dtype, seqs=_log_int(rng, 1, max(1, min(64, room // max_len))), max_len=max_len,
                    channels=channels, n_state=n_state, groups=groups, softplus=rng.random() < 0.8,
                    gate=rng.random() < 0.7, first=rng.random() < 0.5, fused=rng.random() < 0.5)
    vocab = _log_int(rng, 1000, 262144)
    return dict(op=op, dtype=dtype, rows=_log_int(rng, 1, min(4096, (1 << 26) // vocab)), vocab=vocab,
                top=rng.choice([0, 1, 5, 8, 20, 32]), masked=rng.random() < 0.3, padded=rng.random() < 0.5)


def _lens(case):
    """The sequences' lengths: the first is the longest; of eight or more, the second is empty."""
    rng = random.Random(case["seqs"] * 1000003 + case["max_len"])
    lens = [case["max_len"]] + [_log_int(rng, 1, case["max_len"]) for _ in range(case["seqs"] - 1)]
    if len(lens) >= 8:
        lens[1] = 0
    return lens


def work(case):
    """What a pass cannot do without."""
    e = SIZES[case["dtype"]]
    if case["op"] == "logprob":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * e + case["rows"] * (12 + 8 * case["top"]), "flops": 6.0 * n}
    C = case["channels"]
    if case["op"] in ("conv", "conv_step"):
        W = case["width"]
        lens = _lens(case) if case["op"] == "conv" else [1] * case["seqs"]
        T, states = sum(lens), (2 if case["op"] == "conv_step" or case["first"] else 1) * len(lens)
        return {"bytes": 2 * T * C * e + states * (W - 1) * C * e + 4 * C * (W + case["bias"]),
                "flops": 2.0 * T * C * (W + 2 * case["silu"])}
    N, G = case["n_state"], case["groups"]
    lens = _lens(case) if case["op"] == "scan" else [1] * case["seqs"]
    T, states = sum(lens), (2 if case["op"] == "step" or case["first"] else 1) * len(lens)
    return {"bytes": T * C * e * (4 if case["gate"] else 3) + 2 * T * G * N * e + states * C * N * 4 + 4 * C * (N + 2),
            "flops": 7.0 * T * C * N}


# ----------------------------------------------------------------------------------------------- inputs
def _normal(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"conv": _prepare_conv, "conv_step": _prepare_conv, "scan": _prepare_scan, "step": _prepare_scan,
            "logprob": _prepare_logprob}[case["op"]](case, gen)


def _packed(case):
    lens = _lens(case)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    return sum(lens), cu, max(lens)


def _prepare_conv(case, gen):
    dt, C, W, B = DTYPES[case["dtype"]], case["channels"], case["width"], case["seqs"]
    s = dict(op=case["op"], weight=_normal(gen, C, W, scale=W ** -0.5), silu=case["silu"],
             bias=_normal(gen, C, scale=0.1) if case["bias"] else None)
    if case["op"] == "conv":
        T, s["cu"], s["max_len"] = _packed(case)
        rows = torch.empty(T, C + (64 if case["fused"] else 0), dtype=dt, device="cuda")  # a projection's rows
        s["x"] = rows[:, :C]
        s["S0"] = _normal(gen, B, W - 1, C, dtype=dt) if case["first"] else None
        s["S"] = torch.empty(B, W - 1, C, dtype=dt, device="cuda")
    else:
        T = B
        s["x"] = torch.empty(T, C, dtype=dt, device="cuda")
        s["S"] = _normal(gen, B, W - 1, C, dtype=dt)
    s["x"].copy_(_normal(gen, T, C))
    s["y"] = torch.empty(T, C, dtype=dt, device="cuda")
    if own:  # what a user's program keeps beside its buffers: the layer's description
        from quantized_linear_attention_gb300 import lq

        s["cfg"] = lq.conv_config(C, W, dt, silu=case["silu"])
    return s


def _prepare_scan(case, gen):
    """Steps of 0.001 to 0.1 and decay rates around 1 to n_state, as such layers start their training with."""
    dt, C, N, G, B = DTYPES[case["dtype"]], case["channels"], case["n_state"], case["groups"], case["seqs"]
    s = dict(op=case["op"], softplus=case["softplus"])
    if case["op"] == "scan":
        T, s["cu"], s["max_len"] = _packed(case)
        s["S0"] = _normal(gen, B, C, N, scale=0.3) if case["first"] else None
        s["S"] = torch.empty(B, C, N, device="cuda")
    else:
        T = B
        s["S"] = _normal(gen, B, C, N, scale=0.3)
    fused = case.get("fused", False)
    if fused:  # x and z side by side, B and C behind the part that dt is projected from
        xz = torch.empty(T, 2 * C, dtype=dt, device="cuda")
        s["x"], s["z"] = xz[:, :C], xz[:, C:]
        rank = -(-C // 16)
        bc = torch.empty(T, rank + 2 * G * N, dtype=dt, device="cuda")
        s["B"], s["C"] = (bc[:, rank + i * G * N:rank + (i + 1) * G * N].unflatten(1, (G, N)) for i in (0, 1))
    else:
        s["x"], s["z"] = (torch.empty(T, C, dtype=dt, device="cuda") for _ in range(2))
        s["B"], s["C"] = (torch.empty(T, G, N, dtype=dt, device="cuda") for _ in range(2))
    s["x"].copy_(_normal(gen, T, C))
    s["z"].copy_(_normal(gen, T, C))
    s["B"].copy_(_normal(gen, T, G, N))
    s["C"].copy_(_normal(gen, T, G, N))
    if not case["gate"]:
        s["z"] = None
    s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(_normal(gen, C, N, scale=0.3))
    s["D"] = 1 + _normal(gen, C, scale=0.2)
    step = torch.exp(torch.rand(C, generator=gen, device="cuda") * math.log(100) + math.log(0.001))
    if case["softplus"]:
        s["bias"] = torch.log(torch.expm1(step))
        s["dt"] = _normal(gen, T, C, scale=0.5, dtype=dt)
    else:
        s["bias"] = None
        s["dt"] = (step * torch.exp(_normal(gen, T, C, scale=0.5))).to(dt)
    s["y"] = torch.empty(T, C, dtype=dt, device="cuda")
    if own:  # what a user's program keeps beside its buffers: the layer's description and a workspace
        from quantized_linear_attention_gb300 import lq

        s["cfg"] = lq.ssm_config(C, N, G, dt, softplus=case["softplus"])
        if case["op"] == "scan":
            s["workspace"] = torch.empty(lq.ssm_workspace_bytes(s["cfg"], B, T, s["max_len"]), dtype=torch.uint8,
                                         device="cuda")
    return s


def _prepare_logprob(case, gen):
    R, V, K = case["rows"], case["vocab"], case["top"]
    wide = -(-V // 64) * 64 if case["padded"] else V
    full = torch.empty(R, wide, dtype=DTYPES[case["dtype"]], device="cuda")
    full.copy_(_normal(gen, R, wide, scale=2.5))
    logits = full[:, :V]
    tokens = torch.randint(0, V, (R,), generator=gen, device="cuda", dtype=torch.int32)
    if case["masked"]:  # a third of the vocabulary is not allowed next
        logits[torch.rand(R, V, generator=gen, device="cuda") < 1 / 3] = -math.inf
    f, i = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    return dict(op="logprob", logits=logits, tokens=tokens, K=K, logprob=torch.empty(R, **f),
                entropy=torch.empty(R, **f), top=torch.empty(R, K, **f) if K else None,
                top_token=torch.empty(R, K, **i) if K else None)


# ------------------------------------------------------------------------------------------------- runs
def run(s):
    if own:
        from quantized_linear_attention_gb300 import lq

        if s["op"] == "conv":
            lq.conv_prefill(s["cfg"], s["x"], s["weight"], s["y"], bias=s["bias"], cu_seqlens=s["cu"],
                            max_len=s["max_len"], S0=s["S0"], S_out=s["S"])
        elif s["op"] == "conv_step":
            lq.conv_decode_step(s["cfg"], s["S"], s["x"], s["weight"], s["y"], bias=s["bias"])
        elif s["op"] == "scan":
            lq.ssm_prefill(s["cfg"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["y"], D=s["D"], z=s["z"],
                           dt_bias=s["bias"], cu_seqlens=s["cu"], max_len=s["max_len"], S0=s["S0"], S_out=s["S"],
                           workspace=s["workspace"])
        elif s["op"] == "step":
            lq.ssm_decode_step(s["cfg"], s["S"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["y"], D=s["D"], z=s["z"],
                               dt_bias=s["bias"])
        else:
            lq.token_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"], top_logprob=s["top"],
                              top_token=s["top_token"])
            return {"logprob": s["logprob"], "entropy": s["entropy"], "top": s["top"], "top_token": s["top_token"]}
        return {"y": s["y"], "S": s["S"]}
    return {"conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_scan, "step": _plain_step,
            "logprob": _plain_logprob}[s["op"]](s)


def _silu(x):
    return x / (1 + torch.exp(-x))


def _ends(s):
    """For each token its sequence, and its place in it."""
    t = torch.arange(s["x"].shape[0], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"][1:], t, right=True)
    return seq, (t - s["cu"][seq]).long()


def _plain_conv(s):
    x, W = s["x"], s["weight"].shape[1]
    B, C = s["S"].shape[0], x.shape[1]
    seq, at = _ends(s)
    before = torch.zeros(B, W - 1, C, device="cuda") if s["S0"] is None else s["S0"].float()
    rows = torch.cat([x.float(), before.view(-1, C)])  # the tokens, then what came before each sequence

    def taps(seq, begin, at):  # the row that holds the input at place `at` of a sequence, from -(W - 1) on
        return torch.where(at >= 0, begin + at, x.shape[0] + seq * (W - 1) + (W - 1) + at)

    back = torch.arange(1 - W, 1, device="cuda")
    begin = s["cu"].long()
    src = taps(seq[:, None], begin[seq][:, None], at[:, None] + back)  # [T, W]
    y = sum(rows[src[:, j]] * s["weight"][:, j] for j in range(W))
    y = y if s["bias"] is None else y + s["bias"]
    last = taps(torch.arange(B, device="cuda")[:, None], begin[:-1, None], (begin[1:] - begin[:-1])[:, None] + back[:-1])
    return {"y": (_silu(y) if s["silu"] else y).to(x.dtype), "S": rows[last].to(x.dtype)}


def _plain_conv_step(s):
    rows = torch.cat([s["S"], s["x"].unsqueeze(1)], dim=1)
    y = torch.einsum("bwc,cw->bc", rows.float(), s["weight"])
    y = y if s["bias"] is None else y + s["bias"]
    s["S"].copy_(rows[:, 1:])
    return {"y": (_silu(y) if s["silu"] else y).to(s["x"].dtype), "S": s["S"]}


def _delta(s):
    v = s["dt"].float()
    v = v if s["bias"] is None else v + s["bias"]
    return torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0) if s["softplus"] else v


def _skip_and_gate(s, y):
    y = y + s["D"] * s["x"].float()
    return (y if s["z"] is None else y * _silu(s["z"].float())).to(s["x"].dtype)


def _recur(a, b):
    """h[t] = a[t] h[t-1] + b[t] along the first axis: pairs of steps joined into one, again and again."""
    T = a.shape[0]
    if T == 1:
        return b
    odd = _recur(a[1::2] * a[0:T - 1:2], a[1::2] * b[0:T - 1:2] + b[1::2])
    h = torch.empty_like(b)
    h[1::2] = odd
    h[0] = b[0]
    torch.mul(a[2::2], odd[:(T - 1) // 2], out=h[2::2])
    h[2::2] += b[2::2]
    return h


def _plain_scan(s):
    """All sequences as one, whose decay is zero where a sequence begins."""
    x, (C, N), B = s["x"].float(), s["A"].shape, s["S"].shape[0]
    G, many = s["B"].shape[1], C // s["B"].shape[1]
    seq, at = _ends(s)
    delta = _delta(s)
    a = torch.exp(delta[..., None] * s["A"])
    b = ((delta * x).view(-1, G, many, 1) * s["B"].float().unsqueeze(2)).view(-1, C, N)
    first = at == 0
    if s["S0"] is not None:
        b += torch.where(first[:, None, None], a * s["S0"][seq], 0)
    a.masked_fill_(first[:, None, None], 0)
    h = _recur(a, b)
    del a, b
    y = (h.view(-1, G, many, N) * s["C"].float().unsqueeze(2)).sum(-1).view(-1, C)
    cu = s["cu"].long()
    last = h[(cu[1:] - 1).clamp(min=0)]
    zero = torch.zeros_like(last) if s["S0"] is None else s["S0"]
    return {"y": _skip_and_gate(s, y), "S": torch.where((cu[1:] > cu[:-1])[:, None, None], last, zero)}


def _plain_step(s):
    (C, N), G = s["A"].shape, s["B"].shape[1]
    delta = _delta(s)
    a = torch.exp(delta[..., None] * s["A"])
    b = ((delta * s["x"].float()).view(-1, G, C // G, 1) * s["B"].float().unsqueeze(2)).view(-1, C, N)
    s["S"].mul_(a).add_(b)
    y = (s["S"].view(-1, G, C // G, N) * s["C"].float().unsqueeze(2)).sum(-1).view(-1, C)
    return {"y": _skip_and_gate(s, y), "S": s["S"]}


def _plain_logprob(s):
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    lse = top + total.log()
    out = {"logprob": x.gather(1, s["tokens"].long()[:, None]).squeeze(1) - lse.squeeze(1),
           "entropy": (total.log() - torch.where(e > 0, e * (x - top), 0).sum(-1, keepdim=True) / total).squeeze(1),
           "top": None, "top_token": None}
    if s["K"]:  # equal logits in the order of their index: one whole number of both
        bits = (x + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
        V = x.shape[1]
        best = torch.topk(order * (1 << 32) + (V - 1 - torch.arange(V, device="cuda")), s["K"], dim=1).values
        at = V - 1 - (best & 0xffffffff)
        out["top"], out["top_token"] = x.gather(1, at) - lse, at.int()
    return out


# ------------------------------------------------------------------------------------------ definitions
def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "conv_step": _exact_conv, "scan": _exact_scan, "step": _exact_scan,
            "logprob": _exact_logprob}[case["op"]](case, s)


def _sequences(case):
    lens = _lens(case) if "max_len" in case else [1] * case["seqs"]
    return [(b, sum(lens[:b]), n) for b, n in enumerate(lens)]


def _exact_conv(case, s):
    """Sequence by sequence: its state and tokens in one piece, tap by tap."""
    W, w = case["width"], s["weight"].double()
    S0 = s["S"] if case["op"] == "conv_step" else s["S0"]
    y = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    S = torch.empty(s["S"].shape, dtype=torch.float64, device="cuda")
    for b, begin, n in _sequences(case):
        line = torch.zeros(W - 1 + n, w.shape[0], dtype=torch.float64, device="cuda")
        if S0 is not None:
            line[:W - 1] = S0[b]
        line[W - 1:] = s["x"][begin:begin + n]
        out = torch.zeros(n, w.shape[0], dtype=torch.float64, device="cuda")
        for j in range(W):
            out.addcmul_(line[j:j + n], w[:, j])
        if s["bias"] is not None:
            out += s["bias"].double()
        y[begin:begin + n] = out * torch.sigmoid(out) if case["silu"] else out
        S[b] = line[n:]
    return {"y": y, "S": S}


def _exact_scan(case, s):
    """Token by token in 64 bits, the sequences side by side."""
    many = case["channels"] // case["groups"]
    S0 = s["S"] if case["op"] == "step" else s["S0"]
    pieces = sorted(_sequences(case), key=lambda p: -p[2])  # those still running are always the first ones
    order = torch.tensor([p[0] for p in pieces], device="cuda")
    begin = torch.tensor([p[1] for p in pieces], device="cuda")
    h = torch.zeros(s["S"].shape, dtype=torch.float64, device="cuda") if S0 is None else S0.double()[order]
    y = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    A, D = s["A"].double(), s["D"].double()
    running = len(pieces)
    for t in range(pieces[0][2]):
        while pieces[running - 1][2] <= t:
            running -= 1
        at = begin[:running] + t
        x, d = s["x"][at].double(), s["dt"][at].double()
        if s["bias"] is not None:
            d = d + s["bias"].double()
        if case["softplus"]:
            d = torch.logaddexp(d, torch.zeros_like(d))
        Bt = s["B"][at].double().repeat_interleave(many, dim=1)
        Ct = s["C"][at].double().repeat_interleave(many, dim=1)
        live = h[:running]
        live.mul_(torch.exp(d[..., None] * A)).addcmul_((d * x)[..., None], Bt)
        o = torch.einsum("bcn,bcn->bc", live, Ct) + D * x
        if s["z"] is not None:
            z = s["z"][at].double()
            o = o * z * torch.sigmoid(z)
        y[at] = o
    S = torch.empty_like(h)
    S[order] = h
    return {"y": y, "S": S}


def _exact_logprob(case, s):
    R, K = case["rows"], case["top"]
    logprob, entropy = (torch.empty(R, dtype=torch.float64, device="cuda") for _ in range(2))
    top = torch.empty(R, K, dtype=torch.float64, device="cuda") if K else None
    for r in range(0, R, 64):
        p = torch.log_softmax(s["logits"][r:r + 64].double(), dim=1)
        logprob[r:r + 64] = p.gather(1, s["tokens"][r:r + 64].long()[:, None])[:, 0]
        entropy[r:r + 64] = torch.special.entr(torch.exp(p)).sum(1)
        if K:
            top[r:r + 64] = p.sort(dim=1, descending=True).values[:, :K]
    return {"logprob": logprob, "entropy": entropy, "top": top, "top_token": None}
