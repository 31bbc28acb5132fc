"""The selection of beam search (lq_beam_select) against a 64-bit sort."""
import numpy as np
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests._generation import beam_reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.bfloat16, torch.float16, torch.float32]
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


def run(logits, scores, n_best, stream=None):
    B, K, V = logits.shape
    s = torch.full((B, n_best), 77.0, device=DEV)
    p, t = (torch.full((B, n_best), -7, dtype=torch.int32, device=DEV) for _ in range(2))
    ws = torch.full((lq.beam_workspace_bytes(B, K, V, n_best),), 255, dtype=torch.uint8, device=DEV)
    lq.beam_select(logits, scores, s, p, t, ws, stream=stream)
    return s, p, t


def check(logits, scores, n_best):
    s, p, t = (x.cpu().numpy() for x in run(logits, scores, n_best))
    s_r, p_r, t_r = beam_reference(logits.double().cpu().numpy(), scores.cpu().numpy(), n_best)
    assert np.array_equal(p, p_r) and np.array_equal(t, t_r), (p, p_r, t, t_r)
    fine = np.isfinite(s_r)
    assert np.array_equal(fine, np.isfinite(s)) and np.array_equal(s[~fine], s_r[~fine])
    # the final rounding to 32 bits, and a row's sum: its terms' 2^-22 each, taken as if all had one sign
    assert np.all(np.abs(s[fine] - s_r[fine]) <= 2.0 ** -24 * np.abs(s_r[fine]) + 2.0 ** -22)


def inputs(seed, B, K, V, dtype, scale=2.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = (torch.randn(B, K, V, generator=g, device=DEV) * scale).to(dtype)
    return logits, -20.0 * torch.rand(B, K, generator=g, device=DEV)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,K,V,M", [(1, 1, 1, 1), (1, 1, 7, 5), (2, 3, 2, 6), (3, 4, 1000, 8), (2, 5, 8192, 10),
                                     (1, 8, 16385, 16), (2, 32, 511, 64), (1, 3, 50257, 33), (1, 2, 131071, 64)])
def test_sizes(dtype, B, K, V, M):
    check(*inputs(B + K + V, B, K, V, dtype), M)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (2, 2), (24, 0), (7, 3)])
def test_rows_of_any_alignment(dtype, pad, offset):
    B, K, V = 2, 3, 9001
    x, s = inputs(9, B, K, V, dtype)
    flat = torch.full((B * K * (V + pad) + offset,), INF, dtype=dtype, device=DEV)  # not read: it would win
    rows = flat[offset:].view(B, K, V + pad)[:, :, :V]
    rows.copy_(x)
    check(rows, s, 12)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_go_to_the_lowest_index(dtype):
    x, s = inputs(10, 2, 4, 20000, dtype)
    x.copy_(x.clamp(-1, 1).round())  # thousands of equal logits
    s[:, 1] = s[:, 0]
    x[:, 1] = x[:, 0]  # equal hypotheses
    check(x, s, 24)
    x.zero_()
    s.fill_(-1.0)
    check(x, s, 64)
    x[:, :, ::2] = -0.0
    check(x, s, 64)


def test_equal_hypotheses_tie_exactly_whatever_their_place():
    """Rows of odd length start at every alignment; equal contents must still give equal sums."""
    x, s = inputs(11, 1, 1, 33333, torch.bfloat16)
    x, s = x.expand(1, 7, 33333).contiguous(), s.expand(1, 7).contiguous()
    sc, p, t = run(x, s, 14)
    assert p.tolist() == [[0, 1, 2, 3, 4, 5, 6] * 2]
    assert bool((t[0, :7] == t[0, 0]).all()) and bool((sc[0, :7] == sc[0, 0]).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_masks(dtype):
    x, s = inputs(12, 4, 3, 5000, dtype)
    x[0, :, 10:] = -INF  # ten tokens left a row
    x[1, 0] = -INF       # a row with nothing left
    x[2, :, 3:] = -INF   # fewer than n_best candidates in all
    x[3] = -INF          # nothing at all
    check(x, s, 16)
    check(x[2:3, :, :16].contiguous(), s[2:3], 48)


@pytest.mark.parametrize("dtype", TYPES)
def test_lowest_values_are_finite(dtype):
    """A mask of the type's lowest value is a logit like any other: rows of nothing else are even."""
    low = torch.finfo(dtype).min
    x, s = inputs(13, 2, 2, 600, dtype)
    x[0, :, 50:] = low
    x[1] = low
    check(x, s, 20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("at", [1e6, 3e7, 1e30])
def test_large_logits(dtype, at):
    x, s = inputs(14, 2, 2, 40000, dtype)
    x[:, 0] += at
    x[:, 1] -= at
    check(x, s, 8)


def test_dead_hypotheses():
    x, s = inputs(15, 5, 4, 700, torch.float32)
    s[0, 1:] = -INF          # the first selection
    s[1] = -INF              # all dead
    s[2, 2] = float("nan")
    x[3, 1, 44] = float("nan")
    x[4, 2, 3] = INF
    got, p, t = (y.cpu().numpy() for y in run(x, s, 8))
    s_r, p_r, t_r = beam_reference(x.double().cpu().numpy(), s.cpu().numpy(), 8)
    # numpy's maximum of a row with a NaN is NaN and of one with +inf is +inf: dead in the reference as well
    assert np.array_equal(p, p_r) and np.array_equal(t, t_r)
    assert np.array_equal(np.isfinite(got), np.isfinite(s_r))


def test_streams_graphs_and_repeats_give_the_same_bits():
    x, s = inputs(16, 3, 4, 40001, torch.bfloat16)
    a = run(x, s, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = run(x, s, 8, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    out = [torch.zeros_like(y) for y in a]
    ws = torch.empty(lq.beam_workspace_bytes(3, 4, 40001, 8), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream(), capture_error_mode="relaxed"):
        lq.beam_select(x, s, *out, ws)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for y, z, w in zip(a, b, out):
        assert torch.equal(y, z) and torch.equal(y, w)


def test_row_offsets_past_32_bits():
    """Rows 2^30 elements apart: the third starts 4.3 GB in."""
    V, stride = 4099, 1 << 30
    x, s = inputs(17, 1, 3, V, torch.bfloat16)
    rows = torch.empty(2 * stride + V, dtype=torch.bfloat16, device=DEV).as_strided((1, 3, V), (3 * stride, stride, 1))
    rows.copy_(x)
    for y, z in zip(run(rows, s, 6), run(x, s, 6)):
        assert torch.equal(y, z)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("first", [1, 2, 4])
@pytest.mark.parametrize("V", [1, 2, 3, 9, 8191, 16385, 33334])
def test_rows_that_start_off_16_bytes(V, first, dtype):
    """Rows are read by 16 bytes, 4 bytes or single elements, whatever their length; what lies between them is not theirs."""
    x, s = inputs(100 + V, 2, 3, V, dtype)
    stride = (V + 8) // 8 * 8 + first
    all_ = torch.full((6 * stride + 16,), float("nan"), dtype=dtype, device=DEV)
    rows = all_[first:].as_strided((2, 3, V), (3 * stride, stride, 1))
    rows.copy_(x)
    check(rows, s, min(7, 3 * V))
