"""Split prompts (lq_la_prefill where a sequence has several segments)."""
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests._generation import D
from tests.test_la_gpu import check, cu_of, inputs, run, workspace

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", [[90, 1, 0, 130, 40], [90, 1, 0, 120, 40]])
def test_plans_that_find_little_to_split(dtype, lens):
    """No max_len and many tokens that belong to no sequence: segments of 128 tokens (bf16: 512), and of the sequences one is
    longer, or none. What follows in the stream may write the bounds at once."""
    used = sum(lens)
    q, k, v, a, S0 = inputs(1, lens, 2, 1, dtype, first=True)
    cfg = lq.la_config(2, 1, dtype)
    wide = [torch.cat([x, torch.full((3000, *x.shape[1:]), float("nan"), dtype=x.dtype, device=DEV)]) for x in (q, k, v, a)]
    n = used + 3000
    ws = workspace(cfg, 5, n, 0)
    assert ws is not None

    def call():
        cu, o, S = cu_of(lens), torch.full((n, 2, D), 77.0, dtype=dtype, device=DEV), torch.full_like(S0, 77.0)
        lq.la_prefill(cfg, *wide, o, cu_seqlens=cu, S0=S0, S_out=S, workspace=ws)
        return cu, o, S

    _, want_o, want_S = call()
    check(q, k, v, a, lens, S0, want_o[:used], want_S)
    assert bool((want_o[used:] == 77.0).all())
    for _ in range(20):
        cu, o, S = call()
        cu.fill_(n)
        assert torch.equal(o, want_o) and torch.equal(S, want_S)
