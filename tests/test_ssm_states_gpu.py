"""Scans of every class of state counts, and what infinities make of them (lq_ssm_prefill, lq_ssm_decode_step)."""
import numpy as np
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests.test_ssm_gpu import INF, TYPES, call, check, f64, inputs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [17, 25, 32])
@pytest.mark.parametrize("lens,ch,G", [([77], 64, 1), ([77], 301, 1), ([1500], 24, 2), ([640, 3, 0, 901], 33, 1), ([120, 40], 2048, 8),
                                       ([2100], 512, 1)])
def test_seventeen_to_thirty_two_states(dtype, N, lens, ch, G):
    """Short, whole and split calls with few and with many channels, which take other shapes of the kernel."""
    check(inputs(N, lens, ch, N, G, dtype), lens, G, dtype, max_len=max(lens))


def positive(a):
    """Inputs whose outputs are sums of terms of one sign: where one is infinite, so is the output."""
    for k in ("x", "dt", "B", "C", "z", "D", "S0"):
        if a[k] is not None:
            a[k].copy_(a[k].abs() + 0.25)
    return a


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("T,ch", [(60, 16), (77, 256), (1300, 24)])
def test_infinite_outputs(dtype, N, T, ch):
    """An infinite x, step or first state makes its channel infinite from there on, and not NaN, where no state is padding."""
    a = positive(inputs(20, [T], ch, N, 1, dtype))
    a["x"][T // 3, 2], a["dt"][T // 2, 3], a["S0"][0, 7, N - 1] = INF, INF, INF
    a["A"][7] = -1e-4  # (the infinite state never decays to 0 times infinity)
    want = torch.zeros(T, ch, dtype=torch.bool, device=DEV)
    want[T // 3:, 2], want[T // 2:, 3], want[:, 7] = True, True, True
    S = torch.empty(1, ch, N, device=DEV)
    cfg = lq.ssm_config(ch, N, 1, dtype)
    call(cfg, a, [T], S, max_len=T)
    assert torch.equal(a["y"] == INF, want) and not bool(torch.isnan(a["y"]).any())
    inf = torch.zeros(1, ch, N, dtype=torch.bool, device=DEV)
    inf[0, 2:4], inf[0, 7, N - 1] = True, True
    assert torch.equal(S == INF, inf) and not bool(torch.isnan(S).any())
    t, one, s = T // 3, torch.empty(1, ch, dtype=dtype, device=DEV), torch.ones(1, ch, N, device=DEV)
    lq.ssm_decode_step(cfg, s, a["x"][t:t + 1], a["dt"][t:t + 1], a["A"], a["B"][t:t + 1], a["C"][t:t + 1], one, D=a["D"],
                       z=a["z"][t:t + 1], dt_bias=a["bias"])
    assert (one[0] == INF).nonzero().flatten().tolist() == [2] and bool((s[0, 2] == INF).all())
    assert not bool(torch.isnan(one).any() or torch.isnan(s).any()) and np.isfinite(np.delete(f64(s)[0], 2, axis=0)).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,ch,N", [(60, 16, 16), (60, 24, 64), (1300, 24, 8)])
def test_an_infinite_x_without_a_skip_term(dtype, T, ch, N):
    """Without D there is no D x: the token of an infinite x has an infinite output too, not 0 times infinity."""
    a = positive(inputs(21, [T], ch, N, 1, dtype, D=False))
    t = T // 3
    a["x"][t, 2] = INF
    want = torch.zeros(T, ch, dtype=torch.bool, device=DEV)
    want[t:, 2] = True
    cfg, S = lq.ssm_config(ch, N, 1, dtype), torch.empty(1, ch, N, device=DEV)
    call(cfg, a, [T], S, max_len=T)
    assert torch.equal(a["y"] == INF, want) and not bool(torch.isnan(a["y"]).any())
    one, s = torch.empty(1, ch, dtype=dtype, device=DEV), torch.ones(1, ch, N, device=DEV)
    lq.ssm_decode_step(cfg, s, a["x"][t:t + 1], a["dt"][t:t + 1], a["A"], a["B"][t:t + 1], a["C"][t:t + 1], one, z=a["z"][t:t + 1],
                       dt_bias=a["bias"])
    assert (one[0] == INF).nonzero().flatten().tolist() == [2] and not bool(torch.isnan(one).any())


@pytest.mark.parametrize("parts", [1, 60])
@pytest.mark.parametrize("step", [0.1, 0.01, 0.001])
def test_long_memories(step, parts):
    """States that remember from ten to thousands of tokens, in one call (split) and in parts, each going on from the one before.

    d is exact (no softplus, no bias). A decay is off by 4 units of 2^-24 for ex2.approx and |d A| times 2.3 for log2 e, its
    product with A and that one's with d; d x B by two and the fma by one. Where a call is split a sum of d in groups of up to
    32 tokens takes the place of its segment's exponents: off by less than 40 + n / 32 times 2^-24 for n of 64 tokens and more,
    which weighs in by at most 1 / e of that (x e^-x) where the segment's tokens are allowed 4 n."""
    T, ch, N, u = 3840, 40, 16, 2.0 ** -24
    a = inputs(22, [T], ch, N, 1, torch.float32, D=False, z=False, bias=False, first=False, plus=False)
    g = torch.Generator(device=DEV).manual_seed(23)
    a["dt"].copy_(step * torch.exp(0.5 * torch.randn(T, ch, generator=g, device=DEV)))
    a["A"].copy_(-0.1 - 1.4 * torch.rand(ch, N, generator=g, device=DEV))
    for k in ("x", "B"):
        a[k].copy_(a[k].abs() + 0.1)  # (of one sign: what errors add up to shows)
    cfg, S = lq.ssm_config(ch, N, 1, torch.float32, softplus=False), torch.zeros(1, ch, N, device=DEV)
    for t in range(0, T, T // parts):
        part = {k: v[t:t + T // parts] if k in ("x", "dt", "B", "C", "y") else v for k, v in a.items()}
        call(cfg, dict(part, S0=S), [T // parts], S, max_len=T // parts)
    d, x, B, A = f64(a["dt"]), f64(a["x"]), f64(a["B"]), f64(a["A"])
    h = np.zeros((ch, N))
    E = np.zeros((ch, N))
    for t in range(T):
        e = d[t][:, None] * A
        add = (d[t] * x[t])[:, None] * B[t]
        E = np.exp(e) * (E + h * (4 + 2.3 * np.abs(e)) * u) + 2 * u * add
        h = np.exp(e) * h + add
        E += u * h
    err = np.abs(f64(S)[0] - h)
    assert np.all(err <= E), float((err / E).max())
