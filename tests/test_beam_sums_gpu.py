"""The log-sum-exps of the selection (lq_beam_select) where a row's sum is hard to hold: rows of very many equal logits."""
import math

import pytest
import torch

from quantized_linear_attention_gb300 import lq

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
