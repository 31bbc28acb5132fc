"""Log probabilities of given tokens, entropies and the most likely tokens (lq_token_logprobs) against 64 bits."""
import numpy as np
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests._layers import logprob_bounds, logprob_reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.bfloat16, torch.float16, torch.float32]
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


def run(x, tokens, n_top, **kw):
    R = x.shape[0]
    lp, H = (torch.full((R,), 77.0, device=DEV) for _ in range(2))
    tl = torch.full((R, n_top), 77.0, device=DEV) if n_top else None
    ti = torch.full((R, n_top), -7, dtype=torch.int32, device=DEV) if n_top else None
    lq.token_logprobs(x, tokens, lp, entropy=H, top_logprob=tl, top_token=ti, **kw)
    return lp, H, tl, ti


def same(got, want, bound):
    nan, inf = np.isnan(want), np.isinf(want)
    assert np.array_equal(np.isnan(got), nan) and np.array_equal(got[inf], want[inf])
    ok = ~nan & ~inf
    assert np.all(np.abs(got[ok] - want[ok]) <= bound[ok]), np.abs(got[ok] - want[ok]).max()


def check(x, tokens, n_top):
    lp, H, tl, ti = (None if t is None else t.cpu().numpy() for t in run(x, tokens, n_top))
    lp_r, H_r, tl_r, ti_r = logprob_reference(x.double().cpu().numpy(), tokens.cpu().numpy(), n_top)
    with np.errstate(invalid="ignore"):
        bl, bH = logprob_bounds(x.shape[1], lp_r, H_r)
        bt, _ = logprob_bounds(x.shape[1], tl_r, H_r[:, None])
    same(lp, lp_r, bl)
    same(H, H_r, bH)
    if n_top:
        same(tl, tl_r, bt)
        assert np.array_equal(ti, ti_r), (ti, ti_r)


def inputs(seed, R, V, dtype, scale=2.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return ((torch.randn(R, V, generator=g, device=DEV) * scale).to(dtype),
            torch.randint(0, V, (R,), generator=g, device=DEV, dtype=torch.int32))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R,V,k", [(1, 1, 1), (2, 1, 0), (1, 7, 5), (3, 33, 32), (5, 1000, 8), (2, 8192, 20), (3, 8193, 1),
                                   (1, 32000, 32), (1, 131071, 20), (200, 5003, 4), (700, 129, 2), (2, 262144, 32),
                                   (1, 1000003, 10)])
def test_sizes(dtype, R, V, k):
    check(*inputs(R + V, R, V, dtype), k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R", [2, 1300])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (2, 2), (24, 0), (7, 3), (0, 7)])
def test_rows_of_any_alignment(dtype, R, pad, offset):
    V = 901
    x, tok = inputs(9, R, V, dtype)
    flat = torch.full((R * (V + pad) + offset + 16,), INF, dtype=dtype, device=DEV)  # not read: it would win
    v = flat[offset:offset + R * (V + pad)].view(R, V + pad)[:, :V]
    v.copy_(x)
    check(v, tok, 6)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [5, 900, 20000, 70001])
def test_ties_go_to_the_lowest_index(dtype, V):
    x, tok = inputs(10, 4, V, dtype)
    x.copy_(x.clamp(-1, 1).round())  # thousands of equal logits
    x[1] = 0.0
    x[2, ::2] = -0.0
    x[3, V // 2:] = x[3].max()
    for k in (1, 3, 32):
        check(x, tok, min(k, V))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [300, 30000, 131071])
def test_rows_in_order(dtype, V):
    """Rising rows: every element is a new maximum. (16-bit types round neighbours to equal values.)"""
    x = torch.linspace(-30, 30, V, device=DEV).to(dtype).repeat(3, 1)
    x[1] = x[1].flip(0)
    x[2, : V // 2] = -INF
    check(x, torch.tensor([0, V - 1, V // 2], dtype=torch.int32, device=DEV), 20)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [40, 5000, 100000])
def test_masks(dtype, V):
    x, tok = inputs(12, 6, V, dtype)
    x[0, 10:] = -INF             # ten tokens left
    x[1] = -INF                  # a row with nothing left
    x[2, : V - 3] = -INF         # three, at the end
    x[3, torch.arange(V, device=DEV) % 7 != 3] = -INF
    x[4] = -INF
    x[4, V // 2] = -3.0          # one
    x[5, :20] = -INF
    tok[0], tok[2], tok[4] = 3, 1, V // 2
    for k in (0, 1, 16, 32):
        check(x, tok, k)


@pytest.mark.parametrize("dtype", TYPES)
def test_lowest_values_are_finite(dtype):
    """A mask of the type's lowest value is a logit like any other: rows of nothing else are even."""
    low = torch.finfo(dtype).min
    x, tok = inputs(13, 3, 600, dtype)
    x[0, 50:] = low
    x[1] = low
    x[2] = low
    x[2, 100:200] = low * 0.75
    tok[0] = 3
    lp, H, tl, ti = run(x, tok, 20)
    assert abs(H[1].item() - np.log(600)) < 1e-5 and abs(lp[1].item() + np.log(600)) < 1e-5
    assert abs(H[2].item() - np.log(100)) < 1e-5 and ti[2].tolist() == list(range(100, 120))
    assert ti[1].tolist() == list(range(20))
    check(x[:1, :50].contiguous(), tok[:1], 20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("at", [1e4, -1e4, 1e30, -1e30])
def test_large_logits(dtype, at):
    x, tok = inputs(14, 3, 4000, dtype)
    x[1:] += at
    check(x, tok, 8)


def test_peaked_rows():
    """Entropies near zero keep an absolute accuracy; a row of one token has none."""
    x, tok = inputs(15, 3, 3000, torch.float32)
    x[0, 7], x[1, 9], tok[0], tok[1] = 40.0, 200.0, 7, 10
    check(x, tok, 5)
    lp, H, _, _ = run(torch.full((1, 1), 3.5, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV), 1)
    assert lp.item() == 0.0 and H.item() == 0.0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [50, 9000, 131072])
def test_rows_without_a_distribution(dtype, V):
    x, tok = inputs(16, 6, V, dtype)
    x[0, V // 3] = NAN
    x[1, V - 1] = INF
    x[2] = -INF
    x[3, 0] = NAN
    x[4, ::2] = INF
    tok[3] = -1
    lp, H, tl, ti = run(x, tok, 9)
    assert bool(torch.isnan(lp[[0, 1, 2, 4]]).all()) and lp[3].item() == 0.0
    assert bool(torch.isnan(H[:5]).all() and torch.isnan(tl[:5]).all() and (ti[:5] == -1).all())
    assert bool(torch.isfinite(lp[5:]).all() and torch.isfinite(H[5:]).all() and torch.isfinite(tl[5:]).all())


def test_tokens_outside_the_vocabulary():
    x, _ = inputs(17, 5, 100, torch.bfloat16)
    lp, _, _, _ = run(x, torch.tensor([-1, 100, 2**31 - 1, -2**31, 99], dtype=torch.int32, device=DEV), 0)
    assert lp[0] == 0 and lp[3] == 0 and bool(torch.isnan(lp[1:3]).all()) and lp[4] < 0


def test_each_output_alone():
    x, tok = inputs(18, 4, 20001, torch.bfloat16)
    lp, H, tl, ti = run(x, tok, 7)
    a, b, c, d = (torch.zeros_like(t) for t in (lp, H, tl, ti))
    lq.token_logprobs(x, tok, a)
    lq.token_logprobs(x, entropy=b)
    lq.token_logprobs(x, top_logprob=c, top_token=d)
    assert torch.equal(a, lp) and torch.equal(b, H) and torch.equal(c, tl) and torch.equal(d, ti)


@pytest.mark.parametrize("R,V", [(3, 40001), (900, 700)])
def test_streams_graphs_and_repeats_give_the_same_bits(R, V):
    x, tok = inputs(19, R, V, torch.bfloat16)
    a = run(x, tok, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = run(x, tok, 8, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    out = [torch.zeros_like(y) for y in a]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream(), capture_error_mode="relaxed"):
        lq.token_logprobs(x, tok, out[0], entropy=out[1], top_logprob=out[2], top_token=out[3])
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for y, z, w in zip(a, b, out):
        assert torch.equal(y, z) and torch.equal(y, w)


def test_row_offsets_past_32_bits():
    """Rows 2^30 elements apart: the third starts 4.3 GB in."""
    V, stride = 4099, 1 << 30
    x, tok = inputs(20, 3, V, torch.bfloat16)
    rows = torch.empty(2 * stride + V, dtype=torch.bfloat16, device=DEV).as_strided((3, V), (stride, 1))
    rows.copy_(x)
    (lp, H, tl, ti), (lp2, H2, tl2, ti2) = run(rows, tok, 6), run(x, tok, 6)
    assert torch.equal(ti, ti2)
    # The two rows' places relative to 16 bytes differ, and with them the order of a sum's terms: either result is within
    # its own bound of the same number, so they are within twice that of each other.
    bl, bH = logprob_bounds(V, lp2.double().cpu().numpy(), H2.double().cpu().numpy())
    bt, _ = logprob_bounds(V, tl2.double().cpu().numpy(), np.zeros(1))
    for y, z, b in ((lp, lp2, bl), (H, H2, bH), (tl, tl2, bt)):
        assert np.all((y - z).abs().cpu().numpy() <= 2 * b)


def test_agrees_with_beam_selection():
    """The first choice of one hypothesis a request is the most likely token, with the same log probability."""
    x, tok = inputs(21, 9, 30011, torch.bfloat16)
    _, _, tl, ti = run(x, tok, 16)
    s, p, t = (torch.empty(9, 16, dtype=d, device=DEV) for d in (torch.float32, torch.int32, torch.int32))
    ws = torch.empty(lq.beam_workspace_bytes(9, 1, 30011, 16), dtype=torch.uint8, device=DEV)
    lq.beam_select(x[:, None], torch.zeros(9, 1, device=DEV), s, p, t, ws)
    assert torch.equal(t, ti)
    # both are within their own errors of the same numbers
    assert float((s - tl).abs().max()) <= 2.0 ** -22 + float(logprob_bounds(30011, tl.cpu().numpy(), np.zeros(1))[0].max())


def test_no_rows():
    e = torch.empty(0, 50, device=DEV)
    lq.token_logprobs(e, torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, device=DEV))
