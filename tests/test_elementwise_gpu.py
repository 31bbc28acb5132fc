"""silu and softplus of the state space layer's calls, each by itself, against 64 bits."""
import numpy as np
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests._layers import half_step, silu, smallest, softplus
from tests.test_conv_gpu import TYPES, f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


def grid(n, lo, hi):
    """n values: half of them even between lo and hi, half by their magnitude from 1e-4."""
    k = n // 4
    v = np.concatenate([np.linspace(lo, hi, n - 2 * k), -np.geomspace(1e-4, -lo, k), np.geomspace(1e-4, hi, k)])
    return torch.tensor(v, dtype=torch.float32, device=DEV)


# An exponential is off by 4 U for ex2.approx (2^-22), 1 for its last fma and 0.05 |x| for the constant of its reduction;
# 1 + e, its reciprocal and the product with x add 1, 2 and 1. Without the reduction (16-bit outputs) the exponent's two
# roundings weigh 1.3 |x| in place of the fma.
def silu_bound(y, x, dtype):
    s = (9 + 0.05 * np.abs(x)) * U if dtype == torch.float32 else (9 + 1.3 * np.abs(x)) * U
    return s * np.abs(y) + (0 if dtype == torch.float32 else half_step(dtype) * (1 + s) * np.abs(y) + smallest(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C", [4096, 4097])
def test_silu_of_a_convolution(dtype, C):
    """Weights of 0 and 1 pass the last input through: y = silu(x)."""
    x = grid(C, -87.0, 80.0).to(dtype)[None].repeat(11, 1)
    w = torch.tensor([0.0, 1.0], device=DEV).repeat(C, 1)
    cfg, y, one = lq.conv_config(C, 2, dtype), torch.empty_like(x), torch.empty_like(x[:2])
    lq.conv_prefill(cfg, x, w, y)
    lq.conv_decode_step(cfg, torch.zeros(2, 1, C, dtype=dtype, device=DEV), x[:2], w, one)
    want = silu(f64(x[0]))
    for got in list(y) + list(one):
        e = np.abs(f64(got) - want)
        assert np.all(e <= silu_bound(want, f64(x[0]), dtype)), float((e / np.maximum(np.abs(want), 1e-38)).max() / U)


def steps(ch, N, dtype, dt, z=None, T=37):
    """y of tokens whose states are d itself: decays of 0, x and B of 1, one C of 1; and the last states."""
    one = lambda *s: torch.ones(*s, dtype=dtype, device=DEV)
    C = torch.zeros(T, 1, N, dtype=dtype, device=DEV)
    C[:, :, 0] = 1.0
    a = dict(x=one(T, ch), dt=dt.to(dtype)[None].repeat(T, 1), A=torch.full((ch, N), -float("inf"), device=DEV), B=one(T, 1, N),
             C=C, z=None if z is None else z.to(dtype)[None].repeat(T, 1))
    cfg, y, S = lq.ssm_config(ch, N, 1, dtype), torch.empty(T, ch, dtype=dtype, device=DEV), torch.empty(1, ch, N, device=DEV)
    ws = torch.empty(max(256, lq.ssm_workspace_bytes(cfg, 1, T, T)), dtype=torch.uint8, device=DEV)
    lq.ssm_prefill(cfg, a["x"], a["dt"], a["A"], a["B"], a["C"], y, z=a["z"], max_len=T, S_out=S, workspace=ws)
    s1, y1 = torch.zeros(1, ch, N, device=DEV), torch.empty(1, ch, dtype=dtype, device=DEV)
    part = {k: v if v is None or k == "A" else v[:1] for k, v in a.items()}
    lq.ssm_decode_step(cfg, s1, part["x"], part["dt"], a["A"], part["B"], part["C"], y1, z=part["z"])
    return torch.cat([y, y1]), torch.cat([S, s1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ch,N", [(4096, 16), (501, 8), (300, 64), (64, 20)])
def test_softplus_of_a_scan(dtype, ch, N):
    """d = softplus(dt). e^-|v| as above; 2 + e, its reciprocal and their product 1, 2 and 1, the polynomial 1.5 and the last
    fma 1: 12 with it, and 0.05 |v|."""
    dt = grid(ch, -86.0, 60.0)
    _, S = steps(ch, N, dtype, dt)
    v = f64(dt.to(dtype))
    want = softplus(v)[:, None]
    e = np.abs(f64(S) - want)
    assert np.all(e <= (12 + 0.05 * np.abs(v))[:, None] * U * want), float((e / want).max() / U)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ch,N", [(4096, 16), (501, 8), (64, 20)])
def test_gate_of_a_scan(dtype, ch, N):
    """y = h silu(z) of states that are read back."""
    z = grid(ch, -80.0, 80.0)
    y, S = steps(ch, N, dtype, torch.linspace(-2, 2, ch, device=DEV), z)
    zv, h = f64(z.to(dtype)), f64(S)[:, :, 0]
    assert np.array_equal(h[0], h[1])
    want = h[0] * silu(zv)
    e = np.abs(f64(y) - want)
    assert np.all(e <= silu_bound(want, zv, dtype) + U * np.abs(want)), float((e / np.maximum(np.abs(want), 1e-38)).max() / U)
