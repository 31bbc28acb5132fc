"""How often bf16 outputs of prompts (lq_la_prefill) are rounded."""
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests._generation import la_reference, rel
from tests.test_la_gpu import f64, inputs, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("lens", [[100], [128], [60, 13, 127]])
@pytest.mark.parametrize("what", ["state", "tokens", "both"])
def test_prompts_of_one_chunk_are_rounded_once(lens, what):
    """The error is that of the final rounding: what goes in before it is good to 2^-16, so that a rounding falls the other way
    for one output in 2^7 or so and costs at most a step there: below 2% of the squares' sum."""
    q, k, v, a, S0 = inputs(1, lens, 4, 2, torch.bfloat16, first=True, half_life=(100.0, 3000.0))
    if what == "state":
        v *= 2.0 ** -6
    elif what == "tokens":
        S0 *= 2.0 ** -8
    o, _ = run(q, k, v, a, lens, S0)
    o_r, _ = la_reference(f64(q), f64(k), f64(v), f64(a), lens, f64(S0))
    once = rel(f64(torch.from_numpy(o_r).to(torch.bfloat16)), o_r)
    assert rel(f64(o), o_r) <= 1.02 * once, rel(f64(o), o_r) / once
