"""The state space layer's calls and token_logprobs write inside their outputs and workspaces only, and refuse through
the binding what they cannot take."""
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests.test_generation_bounds_gpu import Guarded

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


def cu_of(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,C,W", [([1], 1, 4), ([5, 0, 200], 33, 2), ([3000, 7], 72, 3), ([2, 1], 1032, 4)])
def test_convolution(dtype, lens, C, W):
    T, n = sum(lens), len(lens)
    x, w = torch.randn(T, C, device=DEV).to(dtype), torch.randn(C, W, device=DEV)
    cfg = lq.conv_config(C, W, dtype)
    y, S = Guarded((T, C), dtype), Guarded((n, W - 1, C), dtype)
    lq.conv_prefill(cfg, x, w, y.t, cu_seqlens=cu_of(lens), S_out=S.t)
    lq.conv_prefill(cfg, x, w, y.t, cu_seqlens=cu_of(lens), S0=S.t, S_out=S.t)
    one = Guarded((n, C), dtype)
    lq.conv_decode_step(cfg, S.t, x[:1].expand(n, C).contiguous(), w, one.t)
    torch.cuda.synchronize()
    assert y.intact() and S.intact() and one.intact()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,ch,N", [([1], 1, 1), ([5, 0, 200], 33, 7), ([3000, 7], 40, 16), ([700], 257, 64), ([2600], 24, 8)])
def test_scan(dtype, lens, ch, N):
    T, n = sum(lens), len(lens)
    r = lambda *s: torch.randn(*s, device=DEV)
    cfg = lq.ssm_config(ch, N, 1, dtype)
    x, dt, B, C = (r(T, *s).to(dtype) for s in ((ch,), (ch,), (1, N), (1, N)))
    A = -r(ch, N).abs()
    y, S = Guarded((T, ch), dtype), Guarded((n, ch, N), torch.float32)
    ws = Guarded((lq.ssm_workspace_bytes(cfg, n, T, 0),), torch.uint8)
    for S0 in (None, S.t):
        lq.ssm_prefill(cfg, x, dt, A, B, C, y.t, cu_seqlens=cu_of(lens), S0=S0, S_out=S.t, workspace=ws.t if len(ws.t) else None)
    one = Guarded((n, ch), dtype)
    pick = lambda t: t[:1].expand(n, *t.shape[1:]).contiguous()
    lq.ssm_decode_step(cfg, S.t, pick(x), pick(dt), A, pick(B), pick(C), one.t)
    torch.cuda.synchronize()
    assert y.intact() and S.intact() and ws.intact() and one.intact()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V,k", [(1, 1, 1), (3, 4097, 32), (700, 50, 5), (1, 70001, 20), (2, 131072, 0)])
def test_logprobs(dtype, R, V, k):
    x = torch.randn(R, V, device=DEV).to(dtype)
    x[0, V // 2:] = -float("inf") if V > 1 else 0.0
    lp, H = Guarded((R,), torch.float32), Guarded((R,), torch.float32)
    tl, ti = Guarded((R, k), torch.float32), Guarded((R, k), torch.int32)
    lq.token_logprobs(x, torch.zeros(R, dtype=torch.int32, device=DEV), lp.t, entropy=H.t, top_logprob=tl.t if k else None,
                      top_token=ti.t if k else None)
    torch.cuda.synchronize()
    assert lp.intact() and H.intact() and tl.intact() and ti.intact()
    assert bool((ti.t >= 0).all() and (ti.t < V).all())


def test_convolution_refusals():
    T, C, W = 40, 64, 4
    cfg = lq.conv_config(C, W, torch.float32)
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device=DEV)
    a = dict(x=z(T, C), weight=z(C, W), y=z(T, C), bias=z(C), cu_seqlens=cu_of([30, 10]), S0=z(2, 3, C), S_out=z(2, 3, C))
    bad = [dict(x=z(T, C + 1)), dict(x=z(T, C).half()), dict(x=torch.zeros(T, C)), dict(x=z(T, 2 * C)[:, ::2]), dict(y=z(T + 1, C)),
           dict(y=a["x"]), dict(weight=z(W, C)), dict(weight=z(C, W).double()), dict(bias=z(C + 1)), dict(S0=z(2, C, 3)),
           dict(S_out=z(1, 3, C)), dict(S0=z(2, 3, C).bfloat16()), dict(cu_seqlens=cu_of([30, 10]).long()),
           dict(cu_seqlens=None), dict(x=z(1, C).expand(T, C)), dict(S_out=z(2, 3, 2 * C)[:, :, ::2])]
    for kw in bad:
        with pytest.raises((ValueError, lq.LQError)):
            lq.conv_prefill(cfg, **{**a, **kw})
    lq.conv_prefill(cfg, **a)
    for kw in [dict(S=z(T, C, 3)), dict(S=z(T, 3, C).half()), dict(x=z(T, C)[:, :32]), dict(y=z(T, C, 1)), dict(bias=z(1))]:
        with pytest.raises((ValueError, lq.LQError)):
            lq.conv_decode_step(cfg, **{**dict(S=z(T, 3, C), x=z(T, C), weight=z(C, W), y=z(T, C)), **kw})
    for w in (1, 5):
        with pytest.raises(lq.LQError):
            lq.conv_prefill(lq.conv_config(C, w, torch.float32), z(T, C), z(C, w), z(T, C))


def test_scan_refusals():
    T, ch, N, G = 3000, 32, 16, 2
    cfg = lq.ssm_config(ch, N, G, torch.float32)
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device=DEV)
    a = dict(x=z(T, ch), dt=z(T, ch), A=z(ch, N), B=z(T, G, N), C=z(T, G, N), y=z(T, ch), D=z(ch), z=z(T, ch), dt_bias=z(ch),
             S0=z(1, ch, N), S_out=z(1, ch, N),
             workspace=torch.empty(lq.ssm_workspace_bytes(cfg, 1, T, T), dtype=torch.uint8, device=DEV))
    bad = [dict(x=z(T, ch + 1)), dict(dt=z(T - 1, ch)), dict(z=z(T, ch).half()), dict(A=z(N, ch)), dict(A=z(ch, N).double()),
           dict(B=z(T, N)), dict(B=z(T, N, G)), dict(C=z(T, G, 2 * N)[:, :, ::2]), dict(C=z(T, 2 * G, N)[:, ::2]), dict(y=a["z"]),
           dict(y=torch.zeros(T, ch)), dict(D=z(ch, 1)), dict(dt_bias=z(ch).half()), dict(S0=z(ch, N)), dict(S_out=z(1, N, ch)),
           dict(S_out=z(1, ch, N).half()), dict(cu_seqlens=cu_of([T]).float()), dict(S_out=a["y"].view(-1)[:ch * N].view(1, ch, N))]
    for kw in bad:
        with pytest.raises((ValueError, lq.LQError)):
            lq.ssm_prefill(cfg, **{**a, **kw})
    lq.ssm_prefill(cfg, **a)
    b = dict(S=z(5, ch, N), x=z(5, ch), dt=z(5, ch), A=z(ch, N), B=z(5, G, N), C=z(5, G, N), y=z(5, ch))
    for kw in [dict(S=z(4, ch, N)), dict(B=z(1, G, N)), dict(y=b["x"]), dict(A=z(ch)), dict(dt=z(5, ch).bfloat16()), dict(D=z(1))]:
        with pytest.raises((ValueError, lq.LQError)):
            lq.ssm_decode_step(cfg, **{**b, **kw})
    for kw in (dict(n_state=65), dict(groups=3)):
        with pytest.raises(lq.LQError):
            c = lq.ssm_config(**{**dict(channels=32, n_state=16, groups=1, dtype=torch.float32), **kw})
            lq._check(lq.load().lq_ssm_decode_step(c, None, 1, *[None] * 10))


def test_logprob_refusals():
    R, V = 4, 100
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device=DEV)
    a = dict(logits=z(R, V), tokens=z(R, d=torch.int32), logprob=z(R), entropy=z(R), top_logprob=z(R, 3), top_token=z(R, 3, d=torch.int32))
    bad = [dict(logits=z(V)), dict(logits=torch.zeros(R, V)), dict(logits=z(R, V).double()), dict(logits=z(R, 2 * V)[:, ::2]),
           dict(logits=z(1, V).expand(R, V)), dict(tokens=z(R, d=torch.int64)), dict(tokens=None), dict(logprob=None),
           dict(logprob=z(R + 1)), dict(entropy=z(R, 1)), dict(top_logprob=None), dict(top_token=None), dict(top_token=z(R, 3)),
           dict(top_logprob=z(R, 4)), dict(top_logprob=z(R, 33), top_token=z(R, 33, d=torch.int32)), dict(entropy=a["logprob"]),
           dict(logits=z(R, 2), tokens=z(R, d=torch.int32))]
    for kw in bad:
        with pytest.raises((ValueError, lq.LQError)):
            lq.token_logprobs(**{**a, **kw})
    with pytest.raises(lq.LQError):
        lq.token_logprobs(z(R, V))
    lq.token_logprobs(**a)
    assert bool(((a["entropy"] - 4.6051702).abs() < 1e-5).all())
