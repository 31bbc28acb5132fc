"""Split scans (lq_ssm_prefill where the plan divides long sequences into segments)."""
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests.test_ssm_gpu import TYPES, compare, cu_of, inputs, reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


def scan(cfg, a, cu, S, ws, max_len=0):
    lq.ssm_prefill(cfg, a["x"], a["dt"], a["A"], a["B"], a["C"], a["y"], D=a["D"], z=a["z"], dt_bias=a["bias"], cu_seqlens=cu,
                   max_len=max_len, S0=a["S0"], S_out=S, workspace=ws)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,ch,N,max_len", [([100] * 64, 256, 16, 0), ([64, 1, 0, 50] * 30, 64, 8, 0),
                                               ([100] * 40, 136, 64, 4000), ([60] * 63 + [1200], 72, 16, 0)])
def test_plans_that_find_little_to_split(dtype, lens, ch, N, max_len):
    """Without max_len, or with one far above the lengths, the plan splits though no sequence (in the last case: one) is
    longer than a segment. What follows in the stream may overwrite every input and read every output at once."""
    a = inputs(1, lens, ch, N, 1, dtype)
    cfg, T = lq.ssm_config(ch, N, 1, dtype), sum(lens)
    with pytest.raises(lq.LQError, match="workspace"):  # (on the host: this call is split)
        scan(cfg, a, cu_of(lens), a["S0"], None, max_len)
    ws = torch.empty(lq.ssm_workspace_bytes(cfg, len(lens), T, max_len), dtype=torch.uint8, device=DEV)
    ref = reference(a, lens, True)
    moved = ("x", "dt", "B", "C", "z", "S0")
    work = {k: v.clone() if k in moved + ("y",) else v for k, v in a.items()}
    cu, S = cu_of(lens), torch.empty_like(a["S0"])

    def call_and_overwrite():
        """The call between a fresh set of inputs and their loss; copies of its outputs."""
        for k in moved:
            work[k].copy_(a[k])
        cu.copy_(good)
        work["y"].fill_(77.0)
        S.fill_(77.0)
        scan(cfg, work, cu, S, ws, max_len)
        y1, S1 = work["y"].clone(), S.clone()
        for k in moved:
            work[k].fill_(float("nan"))
        cu.fill_(T)
        ws.fill_(255)
        return y1, S1

    good = cu.clone()
    y, S1 = call_and_overwrite()
    compare(y, S1, ref, dtype)
    for _ in range(10):
        y2, S2 = call_and_overwrite()
        assert torch.equal(y, y2) and torch.equal(S1, S2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream(), capture_error_mode="relaxed"):
        y2, S2 = call_and_overwrite()
    for _ in range(5):
        y2.fill_(5.0)
        S2.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(S1, S2)
