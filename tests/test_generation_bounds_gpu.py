"""The generation calls write inside their outputs and workspaces only: guard regions on both sides of each."""
import pytest
import torch

from quantized_linear_attention_gb300 import lq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
D, GUARD = 128, 4096  # bytes on each side


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


class Guarded:
    """A tensor between two regions of a fixed byte."""

    def __init__(self, shape, dtype):
        n = torch.empty(0, dtype=dtype).element_size()
        for s in shape:
            n *= s
        self.raw = torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device=DEV)
        self.t = self.raw[GUARD:GUARD + n].view(dtype).view(shape)

    def intact(self):
        return bool((self.raw[:GUARD] == 0xA5).all() and (self.raw[-GUARD:] == 0xA5).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("lens", [[1], [5, 0, 200], [129, 127], [3000, 7], [2600]])
def test_prompts(dtype, lens):
    T, H, K = sum(lens), 3, 1
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = (torch.randn(T, n, D, generator=g, device=DEV).to(dtype) for n in (K, K, H))
    a = torch.rand(T, H, generator=g, device=DEV)
    cfg = lq.la_config(H, K, dtype)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    o, S = Guarded((T, H, D), dtype), Guarded((len(lens), H, D, D), torch.float32)
    n = lq.la_workspace_bytes(cfg, len(lens), T, max(lens))
    ws = Guarded((n,), torch.uint8)
    lq.la_prefill(cfg, q, k, v, a, o.t, cu_seqlens=cu, max_len=max(lens), S_out=S.t, workspace=ws.t if n else None)
    lq.la_prefill(cfg, q, k, v, a, o.t, cu_seqlens=cu, max_len=max(lens), S0=S.t, S_out=S.t,
                  workspace=ws.t if n else None)
    torch.cuda.synchronize()
    assert o.intact() and S.intact() and ws.intact()
    step = Guarded((len(lens), H, D), dtype)
    lq.la_decode_step(cfg, S.t, *(x[:len(lens)].contiguous() for x in (q, k, v, a)), step.t) if T >= len(lens) else None
    torch.cuda.synchronize()
    assert step.intact() and S.intact()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,K,V,M", [(1, 1, 1, 1), (3, 5, 4097, 10), (2, 32, 700, 64), (1, 2, 70001, 33)])
def test_selection(dtype, B, K, V, M):
    x, s = torch.randn(B, K, V, device=DEV).to(dtype), torch.zeros(B, K, device=DEV)
    x[0, 0, V // 2:] = -float("inf")
    M = min(M, K * V)
    best, parent, token = Guarded((B, M), torch.float32), Guarded((B, M), torch.int32), Guarded((B, M), torch.int32)
    ws = Guarded((lq.beam_workspace_bytes(B, K, V, M),), torch.uint8)
    lq.beam_select(x, s, best.t, parent.t, token.t, ws.t)
    torch.cuda.synchronize()
    assert best.intact() and parent.intact() and token.intact() and ws.intact()
    assert bool((parent.t >= 0).all() and (parent.t < K).all() and (token.t >= 0).all() and (token.t < V).all())


@pytest.mark.parametrize("kda", [False, True])
def test_reordering(kda):
    cfg = lq.config(window=5, n_comp=3, kda=kda)
    n = 2 * 3 * 4
    state = Guarded((lq.state_bytes(cfg, n),), torch.uint8)
    lq.state_init(cfg, state.t, n, torch.randn(n, D, D, device=DEV))
    par = torch.tensor([[1, 1, 3, 0]] * 3, dtype=torch.int32, device=DEV)
    lq.state_reorder(cfg, state.t, n, par, outer=2)
    S = Guarded((n, D, D), torch.float32)
    lq.fp32_state_reorder(S.t, par, outer=2)
    torch.cuda.synchronize()
    assert state.intact() and S.intact() and lq.get_status(state.t)[0] == lq.OK
