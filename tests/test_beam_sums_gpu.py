"""The log-sum-exps of the selection (lq_beam_select) where a row's sum is hard to hold (very many equal logits) or
decides between beams (nearly equal scores)."""
import math

import numpy as np
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests._generation import beam_reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


def select(logits, scores, n_best):
    B, K, V = logits.shape
    s = torch.full((B, n_best), 77.0, device=DEV)
    p, t = (torch.full((B, n_best), -7, dtype=torch.int32, device=DEV) for _ in range(2))
    ws = torch.full((lq.beam_workspace_bytes(B, K, V, n_best),), 255, dtype=torch.uint8, device=DEV)
    lq.beam_select(logits, scores, s, p, t, ws)
    return s, p, t


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("V", [2**24 - 1, 2**24, 2**24 + 1000, 2**25 + 3, 2**26 + 1])
@pytest.mark.parametrize("value", [0.0, -3.0, 3.0e7])
def test_even_rows_of_many_tokens(V, dtype, value):
    """Every token of an even row scores -log V, whatever the logits' value: terms of 1 each, 2^24 and more of them."""
    if dtype == torch.float16:
        value = min(value, 60000.0)
    x = torch.full((1, 1, V), value, dtype=dtype, device=DEV)
    s, p, t = select(x, torch.zeros(1, 1, device=DEV), 5)
    assert t.tolist() == [[0, 1, 2, 3, 4]] and p.tolist() == [[0] * 5]
    # the final rounding to 32 bits, and a row's sum: its terms' 2^-22 each, taken as if all had one sign
    want = -math.log(V)
    assert all(abs(x - want) <= 2.0 ** -24 * abs(want) + 2.0 ** -22 for x in s[0].tolist()), (s, want)


def close_rows(kind, seed, K, V, dtype):
    """Rows of which the best token's score hangs on the row's sum."""
    g = torch.Generator().manual_seed(seed)
    if kind == "peak":  # nearly all of a row's weight on one token
        x = torch.randn(1, K, V, generator=g)
        x[0, torch.arange(K), torch.randint(0, V, (K,), generator=g)] = 11.0 + torch.rand(K, generator=g)
    elif kind == "even":  # a thread's terms round alike
        x = (torch.rand(1, K, 1, generator=g) * 6).expand(1, K, V).contiguous()
    elif kind == "large":
        x = 3.0e6 + 2.5 * torch.randn(1, K, V, generator=g)
    else:
        x = 2.5 * torch.randn(1, K, V, generator=g)
    return x.to(dtype)


def close_scores(loss, seed, gap):
    """fp32 scores that make up for the rows' sums: the best candidates lie `gap` apart (to a tenth) or a step of fp32 more."""
    s, last = np.zeros(len(loss), np.float32), -np.inf
    for i, b in enumerate(np.random.default_rng(seed).permutation(len(loss))):
        least = last + 0.9 * gap + (loss[b] - loss[0])
        s[b] = loss[b] - loss[0] + gap * i
        if s[b] < least:  # the next fp32 number that is not below it
            s[b] = least
            s[b] = np.nextafter(s[b], np.float32(np.inf)) if s[b] < least else s[b]
        last = s[b] - (loss[b] - loss[0])
    return s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("kind", ["peak", "even", "spread", "large"])
@pytest.mark.parametrize("gap", [5e-8, 4e-9])
@pytest.mark.parametrize("V", [600, 40001])
def test_nearly_equal_hypotheses_keep_their_order(V, gap, kind, dtype):
    """Eight beams whose best candidates lie within a few 1e-8, or 1e-9, of one another: the order is the exact scores'."""
    if kind == "large" and dtype == torch.float16:
        pytest.skip("past fp16")
    K = 8
    for seed in range(3):
        x = close_rows(kind, seed, K, V, dtype)
        y = x.double().numpy()[0]
        top = y.max(axis=1)
        loss = np.log(np.exp(y - top[:, None]).sum(axis=1))
        s = torch.from_numpy(close_scores(loss, seed, gap))[None]
        got, p, t = (z.cpu().numpy() for z in select(x.to(DEV), s.to(DEV), 12))
        want, p_r, t_r = beam_reference(x.double().numpy(), s.numpy(), 12)
        assert np.array_equal(p, p_r) and np.array_equal(t, t_r), (p, p_r, t, t_r)
        assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -22)


def test_more_ties_than_the_list_holds_in_rows_of_different_sums():
    """2,304 candidates that tie but for 4e-9 a beam."""
    K, V = 3, 200000
    x = torch.tensor([0.3, 1.7, 2.9])[None, :, None].expand(1, K, V).contiguous()
    s = torch.tensor([[0.0, 8e-9, 4e-9]])
    got, p, t = (z.cpu().numpy() for z in select(x.to(DEV), s.to(DEV), 64))
    assert np.array_equal(p, np.full((1, 64), 1)) and np.array_equal(t, np.arange(64)[None])


def test_equal_rows_tie_exactly_beside_nearly_equal_ones():
    """Beams 0 and 2 are the same, beam 1 is 1e-9 better: it comes first, the others by their index."""
    V = 30011
    x = close_rows("peak", 5, 1, V, torch.bfloat16).expand(1, 3, V).contiguous()
    y = x.double().numpy()[0]
    x[0, 1, 7] = -30.0  # another row, of nearly the same sum
    z = x.double().numpy()[0]
    d = np.log(np.exp(z).sum(axis=1)) - np.log(np.exp(y).sum(axis=1))
    s = torch.tensor([[0.0, d[1] + 1e-9, 0.0]], dtype=torch.float32)
    got, p, t = (w.cpu().numpy() for w in select(x.to(DEV), s.to(DEV), 3))
    want, p_r, t_r = beam_reference(x.double().numpy(), s.numpy(), 3)
    assert p_r.tolist() == [[1, 0, 2]]
    assert np.array_equal(p, p_r) and np.array_equal(t, t_r)
