"""What the Python binding of the generation calls refuses before a kernel runs: always by ValueError or LQError."""
import pytest
import torch

from quantized_linear_attention_gb300 import lq

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


def select(**kw):
    B, K, V, M = 2, 3, 100, 4
    a = dict(logits=torch.zeros(B, K, V, device=DEV), scores=torch.zeros(B, K, device=DEV),
             out_scores=torch.full((B, M), 7.0, device=DEV), out_parent=torch.zeros(B, M, dtype=torch.int32, device=DEV),
             out_token=torch.zeros(B, M, dtype=torch.int32, device=DEV),
             workspace=torch.empty(lq.beam_workspace_bytes(B, K, V, M), dtype=torch.uint8, device=DEV))
    a.update(kw)
    lq.beam_select(**a)
    return a


def test_selection():
    bad = [dict(workspace=None), dict(workspace=torch.empty(64, dtype=torch.uint8, device=DEV)),
           dict(scores=torch.zeros(2, 4, device=DEV)), dict(scores=torch.zeros(2, 3, dtype=torch.float64, device=DEV)),
           dict(out_scores=torch.zeros(4, device=DEV)), dict(out_scores=torch.zeros(2, 5, device=DEV)),
           dict(out_parent=torch.zeros(2, 4, device=DEV)), dict(logits=torch.zeros(3, 100, device=DEV)),
           dict(logits=torch.zeros(2, 3, 100)), dict(logits=torch.zeros(2, 3, 100, dtype=torch.float64, device=DEV)),
           dict(logits=torch.zeros(2, 3, 200, device=DEV)[:, :, ::2]), dict(logits=torch.zeros(1, 1, 100, device=DEV).expand(2, 3, 100))]
    for kw in bad:
        with pytest.raises((ValueError, lq.LQError)):
            select(**kw)
    assert bool((select()["out_scores"] < 0).all())


def test_prompts():
    cfg = lq.la_config(2, 1, torch.float32)
    T = 3000
    mk = lambda n: torch.zeros(T, n, 128, device=DEV)
    a = dict(q=mk(1), k=mk(1), v=mk(2), alpha=torch.ones(T, 2, device=DEV), o=mk(2), max_len=T,
             workspace=torch.empty(lq.la_workspace_bytes(cfg, 1, T, T), dtype=torch.uint8, device=DEV))
    bad = [dict(workspace=None), dict(workspace=a["workspace"][:256]), dict(q=mk(2)), dict(o=mk(2)[:10]), dict(k=a["k"].half()),
           dict(v=a["v"].cpu()), dict(alpha=a["alpha"].double()), dict(alpha=a["alpha"][:, :1]), dict(q=torch.zeros(T, 128, device=DEV)),
           dict(S0=torch.zeros(128, 128, device=DEV)), dict(S_out=torch.zeros(1, 2, 128, 128, dtype=torch.float64, device=DEV)),
           dict(cu_seqlens=torch.tensor([0, T], device=DEV)), dict(o=a["v"])]
    for kw in bad:
        with pytest.raises((ValueError, lq.LQError)):
            lq.la_prefill(cfg, **{**a, **kw})
    lq.la_prefill(cfg, **a)
    assert bool((a["o"] == 0).all())
