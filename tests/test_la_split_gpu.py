"""Split prompts (lq_la_prefill where a sequence has several segments): in place, captured in a graph, on another stream,
from states at any 16-byte address, and plans that find little to split."""
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


LENS = [2900, 64, 0, 1, 3500]


@pytest.mark.parametrize("dtype", TYPES)
def test_in_place(dtype):
    """Last states that replace the first ones: every segment still starts from what the call found."""
    q, k, v, a, S0 = inputs(2, LENS, 1, 1, dtype, first=True, half_life=(20.0, 20000.0))
    o, S = run(q, k, v, a, LENS, S0)
    check(q, k, v, a, LENS, S0, o, S)
    same = S0.clone()
    o2, _ = run(q, k, v, a, LENS, same, S_out=same)
    assert torch.equal(o, o2) and torch.equal(S, same)
    again = S0.clone()  # the states are read where nothing is asked of them afterwards, too
    o3, none = run(q, k, v, a, LENS, again, S_out=None)
    assert none is None and torch.equal(o, o3) and torch.equal(again, S0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_in_a_graph(dtype, in_place):
    """Three or four launches, two of them set up while the one before runs."""
    q, k, v, a, S0 = inputs(3, LENS, 1, 1, dtype, first=True)
    want_o, want_S = run(q, k, v, a, LENS, S0)
    cfg, cu, B, T = lq.la_config(1, 1, dtype), cu_of(LENS), len(LENS), sum(LENS)
    ws, o, S = workspace(cfg, B, T, max(LENS)), torch.zeros_like(want_o), torch.zeros_like(want_S)
    first = S if in_place else S0.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream(), capture_error_mode="relaxed"):
        lq.la_prefill(cfg, q, k, v, a, o, cu_seqlens=cu, max_len=max(LENS), S0=first, S_out=S, workspace=ws)
    for _ in range(3):
        ws.fill_(255)
        o.fill_(77.0)
        first.copy_(S0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want_o) and torch.equal(S, want_S)
    first.copy_(S0)
    q.copy_(q.flip(0))  # other inputs, in the same buffers
    first.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    other_o, other_S = run(q, k, v, a, LENS, S0 * 0.5)
    assert torch.equal(o, other_o) and torch.equal(S, other_S)


@pytest.mark.parametrize("dtype", TYPES)
def test_on_another_stream_and_from_any_address(dtype):
    q, k, v, a, S0 = inputs(4, LENS, 1, 1, dtype, first=True)
    want_o, want_S = run(q, k, v, a, LENS, S0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, S = run(q, k, v, a, LENS, S0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want_o) and torch.equal(S, want_S)
    raw = torch.empty(2, S0.numel() + 4, device=DEV)
    first, last = (raw[i, 4:].view(S0.shape) for i in range(2))
    assert first.data_ptr() % 32 == 16
    first.copy_(S0)
    o, _ = run(q, k, v, a, LENS, first, S_out=last)
    assert torch.equal(o, want_o) and torch.equal(last, want_S)
    o, _ = run(q, k, v, a, LENS, first, S_out=first)
    assert torch.equal(o, want_o) and torch.equal(first, want_S)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("length", [2049, 2560, 2561, 4096, 4097])
def test_lengths_about_whole_segments(dtype, length):
    lens = [length, 7]
    q, k, v, a, S0 = inputs(length, lens, 1, 1, dtype, first=length % 2 == 0)
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)
