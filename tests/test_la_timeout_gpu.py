"""The bounded waits of chunked prompts (lq_la_prefill, bf16), made to run out (no GPU fault is provoked).

The test hook lq_debug_set_wait shortens this thread's bound to 1 ms and makes the kernel announce 16 bytes more to a
chunk's barrier than it copies: every copy lands, the barrier never completes, and the waits give up. The outputs and last
states must then be NaN, and the context stays usable.
"""
import time

import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests.test_la_gpu import check, inputs, run

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(autouse=True)
def _hook_off():
    lq.load()
    torch.cuda.set_device(DEV)
    lq.debug_set_wait(0, 0, 0)
    yield
    lq.debug_set_wait(0, 0, 0)


def late(*args, **kw):
    lq.debug_set_wait(1_000_000, 16, 0)
    t0 = time.monotonic()
    out = run(*args, **kw)
    torch.cuda.synchronize()
    lq.debug_set_wait(0, 0, 0)
    assert time.monotonic() - t0 < 5.0
    return out


@pytest.mark.parametrize("lens", [[20], [128], [256], [300, 128, 0, 14], [900]])
def test_waits_that_run_out_leave_nan(lens):
    q, k, v, a, S0 = inputs(1, lens, 2, 1, torch.bfloat16, first=True)
    o, S = late(q, k, v, a, lens, S0)
    assert bool(o.isnan().all())
    for b, n in enumerate(lens):
        assert bool(S[b].isnan().all()) if n else torch.equal(S[b], S0[b])
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)


def test_states_in_place():
    q, k, v, a, S0 = inputs(2, [200], 2, 1, torch.bfloat16, first=True)
    S = S0.clone()
    o, _ = late(q, k, v, a, [200], S, S_out=S)
    assert bool(o.isnan().all()) and bool(S.isnan().all())
    S.copy_(S0)
    o, _ = run(q, k, v, a, [200], S, S_out=S)
    check(q, k, v, a, [200], S0, o, S)


def test_split_prompts_go_token_by_token():
    """Where the first pass gives up there is no state between the segments, so the sequence is taken token by token."""
    lens = [2900, 30]
    q, k, v, a, S0 = inputs(3, lens, 1, 1, torch.bfloat16, first=True)
    o, S = late(q, k, v, a, lens, S0)
    check(q[:2900], k[:2900], v[:2900], a[:2900], lens[:1], S0[:1], o[:2900], S[:1])
    assert bool(o[2900:].isnan().all()) and bool(S[1].isnan().all())
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)
