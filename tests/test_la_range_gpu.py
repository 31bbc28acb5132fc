"""Prompts (lq_la_prefill) at the ends of fp32's range: values, states and decays that are large, infinite or not a number,
compared with the 64-bit recurrence entry by entry, the sign of every infinity included."""
import numpy as np
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests._generation import D, la_reference, output_bound, rel, state_bound
from tests.test_la_gpu import f64, inputs, run

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.bfloat16, torch.float16, torch.float32]
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


def same(got, want, bound):
    """NaN, inf and -inf where the reference has them; the finite entries within `bound` of it."""
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isposinf(got), np.isposinf(want)) and np.array_equal(np.isneginf(got), np.isneginf(want))
    fine = np.isfinite(want)
    assert rel(got[fine], want[fine]) <= bound, rel(got[fine], want[fine])


def check(q, k, v, a, lens, S0, o, S):
    o_r, S_r = la_reference(f64(q), f64(k), f64(v), f64(a), lens, None if S0 is None else f64(S0))
    n = max(lens)
    same(f64(S), S_r, state_bound(n))
    same(f64(o), o_r, output_bound(q.dtype, n))


@pytest.mark.parametrize("dtype,n", [(torch.float32, 5), (torch.float32, 90), (torch.bfloat16, 11), (torch.bfloat16, 200)])
@pytest.mark.parametrize("decay", [0.4, 0.05])
def test_large_finite_values(dtype, n, decay):
    """Values near 1e37: kept divided by the product of a few decays they would pass fp32's largest number."""
    q, k, v, a, _ = inputs(1, [n], 2, 1, dtype)
    v *= 1e36
    a.fill_(decay)
    o, S = run(q, k, v, a, [n])
    check(q, k, v, a, [n], None, o, S)


@pytest.mark.parametrize("n", [6, 60])
def test_large_states_and_queries(n):
    """States near 1e35 that decay at once and queries near 150: divided by the decays the output's sum would pass the
    largest number."""
    q, k, v, a, _ = inputs(2, [n], 2, 1, torch.float32)
    q *= 150
    a.fill_(0.3)
    S0 = 1e35 * torch.randn(1, 2, D, D, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    o, S = run(q, k, v, a, [n], S0)
    check(q, k, v, a, [n], S0, o, S)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [INF, -INF])
@pytest.mark.parametrize("what", ["v", "k", "S0"])
def test_infinite_states_stay_infinite(dtype, value, what):
    """An infinity keeps its sign from token to token, whatever the decays; it becomes NaN only as the recurrence says."""
    lens = [40, 9, 130]
    q, k, v, a, S0 = inputs(3, lens, 2, 2, dtype, first=True)
    for b, at in enumerate((3, 40 + 2, 49 + 50)):
        if what == "S0":
            S0[b, 1, 17, 5] = value
        else:
            {"v": v, "k": k}[what][at, 1, 5] = value
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("kind", ["zero", "nan", "infinite", "above one", "negative"])
def test_odd_decays_beside_infinite_states(dtype, kind):
    lens = [50]
    q, k, v, a, S0 = inputs(4, lens, 2, 2, dtype, first=True)
    k[3, 0, 5] = INF
    if kind == "above one":
        a[10:16] = 1.7
    elif kind == "negative":
        a[10:31] *= -1
    else:
        a[20, 1] = {"zero": 0.0, "nan": float("nan"), "infinite": INF}[kind]
        if kind == "zero":
            a[20, 0] = 0.0
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)


LONG = 2900  # one head: split in every type


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("first", [False, True])
def test_split_prompts_whose_decays_pass_the_largest_number(dtype, first):
    """Decays of 2: their product over a segment is infinite, and the state that it multiplies is zero until the last tokens."""
    q, k, v, a, _ = inputs(5, [LONG], 1, 1, dtype)
    v[:LONG - 9] = 0
    a.fill_(2.0)
    S0 = torch.zeros(1, 1, D, D, device=DEV) if first else None
    o, S = run(q, k, v, a, [LONG], S0)
    check(q, k, v, a, [LONG], S0, o, S)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [INF, -INF, float("nan")])
@pytest.mark.parametrize("what", ["v", "k", "S0", "alpha"])
def test_infinities_in_split_prompts(dtype, value, what):
    """Two split sequences and a short one between; the infinity is in the first, in its second segment or before it."""
    lens = [LONG, 30, LONG - 300]
    q, k, v, a, S0 = inputs(6, lens, 1, 1, dtype, first=True)
    clean_o, clean_S = run(q, k, v, a, lens, S0)
    if what == "S0":
        S0[0, 0, 17, 5] = value
    elif what == "alpha":
        a[700, 0] = value
    else:
        {"v": v, "k": k}[what][700, 0, 5] = value
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)
    assert torch.equal(o[LONG:], clean_o[LONG:]) and torch.equal(S[1:], clean_S[1:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["negative", "above one", "zeros", "tiny"])
def test_odd_decays_in_split_prompts(dtype, kind):
    lens = [LONG, 30]
    q, k, v, a, S0 = inputs(7, lens, 1, 1, dtype, first=True, half_life=(20.0, 20000.0))
    if kind == "negative":
        a[::3] *= -1
    elif kind == "above one":
        a[::2] = 1.003
    elif kind == "zeros":
        a[::700] = 0
    else:
        a[::700] = 1e-42
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)


@pytest.mark.parametrize("dtype", TYPES)
def test_split_prompts_of_large_finite_values(dtype):
    """Values near 1e36 (2e4 in fp16) that decay fast, in every segment."""
    q, k, v, a, S0 = inputs(8, [LONG], 1, 1, dtype, first=True)
    v *= 4000 if dtype == torch.float16 else 1e36
    a.fill_(0.3)
    o, S = run(q, k, v, a, [LONG], S0)
    fits = np.abs(la_reference(f64(q), f64(k), f64(v), f64(a), [LONG], f64(S0))[0]).max() < torch.finfo(dtype).max
    assert fits
    check(q, k, v, a, [LONG], S0, o, S)


@pytest.mark.parametrize("dtype", TYPES)
def test_states_in_place_of_split_prompts_with_an_infinity(dtype):
    q, k, v, a, S0 = inputs(9, [LONG], 1, 1, dtype, first=True)
    k[700, 0, 5] = INF
    S = S0.clone()
    o, _ = run(q, k, v, a, [LONG], S, S_out=S)
    check(q, k, v, a, [LONG], S0, o, S)


@pytest.mark.parametrize("lens", [[100], [300]])
@pytest.mark.parametrize("what", ["state", "scores"])
def test_chunked_products_that_pass_the_largest_number_before_they_decay(lens, what):
    """bf16: S q, or q k, is past fp32's largest number, the decays in front of it are not."""
    q, k, v, a, S0 = inputs(10, lens, 2, 1, torch.bfloat16, first=True)
    a.fill_(0.5)
    a[7::16] = 1e-12
    q *= 1e12
    if what == "state":
        S0 *= 1e30
        v[:7] = 0
        q[:7] = 0
    else:
        k[7::16] *= 1e30
        q[7::16] = 0
        v *= 1e-20
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [INF, -INF, float("nan")])
@pytest.mark.parametrize("n", [10, 100, 300])
def test_infinite_queries(dtype, value, n):
    q, k, v, a, S0 = inputs(11, [n], 2, 2, dtype, first=True)
    q[n // 2, 1, 5] = value
    q[n - 1, 0, 9] = value
    o, S = run(q, k, v, a, [n], S0)
    check(q, k, v, a, [n], S0, o, S)


@pytest.mark.parametrize("n", [100, 300])
def test_infinite_outputs_of_states_in_place(n):
    """The tokens are taken again from the first state, which must still be there."""
    q, k, v, a, S0 = inputs(12, [n], 2, 2, torch.bfloat16, first=True)
    q[n - 1, 0, 9] = INF
    S = S0.clone()
    o, _ = run(q, k, v, a, [n], S, S_out=S)
    check(q, k, v, a, [n], S0, o, S)


def test_infinities_next_to_a_ragged_end_change_nothing_there():
    """The tokens behind a prompt's last chunk are another prompt's: its infinite queries leave the first one's bits."""
    lens = [70, 80]
    q, k, v, a, S0 = inputs(13, lens, 2, 2, torch.bfloat16, first=True)
    clean_o, clean_S = run(q, k, v, a, lens, S0)
    q[70:, :, 3] = INF
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)
    assert torch.equal(o[:70], clean_o[:70]) and torch.equal(S[0], clean_S[0])
