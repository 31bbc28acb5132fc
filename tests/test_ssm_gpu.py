"""The selective state space scan (lq_ssm_prefill, lq_ssm_decode_step) against the recurrence in 64 bits."""
import numpy as np
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests._layers import half_step, smallest, ssm_reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.bfloat16, torch.float16, torch.float32]
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def cu_of(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)


def rows(t, pad, offset, fill=float("nan")):
    """The same values with `pad` elements between tokens, `offset` elements into the allocation."""
    T, n = t.shape[0], int(np.prod(t.shape[1:]))
    flat = torch.full((T * (n + pad) + offset,), fill, dtype=t.dtype, device=DEV)
    v = flat[offset:].view(T, n + pad)[:, :n].unflatten(1, t.shape[1:])
    v.copy_(t)
    return v


def inputs(seed, lens, ch, N, G, dtype, D=True, z=True, bias=True, first=True, plus=True, pad=0, offset=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    T, n = sum(lens), len(lens)
    put = lambda t: rows(t.to(dtype), pad, offset)
    step = torch.exp(torch.rand(ch, generator=g, device=DEV) * np.log(100) + np.log(0.001))
    return dict(x=put(r(T, ch)), dt=put(0.5 * r(T, ch) if plus else (step * torch.exp(0.5 * r(T, ch)))),
                A=-torch.arange(1, N + 1, device=DEV) * torch.exp(0.3 * r(ch, N)), B=put(r(T, G, N)), C=put(r(T, G, N)),
                y=rows(torch.zeros(T, ch, dtype=dtype, device=DEV), pad, offset, 5.0), D=r(ch) if D else None,
                z=put(r(T, ch)) if z else None, bias=torch.log(torch.expm1(step)) if bias and plus else None,
                S0=r(n, ch, N) if first else None)


def call(cfg, a, lens, S, max_len=0, cu=None, **kw):
    n = len(lens)
    ws = torch.full((lq.ssm_workspace_bytes(cfg, n, a["x"].shape[0], max_len),), 255, dtype=torch.uint8, device=DEV)
    lq.ssm_prefill(cfg, a["x"], a["dt"], a["A"], a["B"], a["C"], a["y"], D=a["D"], z=a["z"], dt_bias=a["bias"],
                   cu_seqlens=cu_of(lens) if cu is None else cu, max_len=max_len, S0=a["S0"], S_out=S,
                   workspace=ws if ws.numel() else None, **kw)


def reference(a, lens, plus, S0=None):
    return ssm_reference(f64(a["x"]), f64(a["dt"]), f64(a["A"]), f64(a["B"]), f64(a["C"]), lens, f64(a["D"]), f64(a["z"]),
                         f64(a["bias"]), f64(a["S0"] if S0 is None else S0), plus)


def compare(y, S, ref, dtype):
    y_r, S_r, Ey, ES = ref
    e = np.abs(f64(y) - y_r)
    assert np.all(e <= half_step(dtype) * (np.abs(y_r) + Ey) + Ey + smallest(dtype)), float((e / (Ey + np.abs(y_r))).max())
    if S is not None:
        e = np.abs(f64(S) - S_r)
        assert np.all(e <= ES), float((e / ES).max())


def check(a, lens, G, dtype, plus=True, max_len=0, in_place=False):
    ch, N = a["A"].shape
    ref = reference(a, lens, plus)
    S = a["S0"] if in_place else torch.full((len(lens), ch, N), 7.0, device=DEV)
    call(lq.ssm_config(ch, N, G, dtype, softplus=plus), a, lens, S, max_len)
    compare(a["y"], S, ref, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,ch,N,G", [([1], 1, 1, 1), ([2, 0, 3], 5, 3, 1), ([40], 130, 16, 1), ([33, 1, 65], 96, 8, 2),
                                         ([50], 100, 12, 4), ([70, 31], 257, 17, 1), ([64], 256, 32, 1),
                                         ([45, 6], 66, 64, 2), ([16, 17, 15, 8, 9, 7], 128, 16, 1), ([100], 24, 33, 8)])
def test_sizes(dtype, lens, ch, N, G):
    check(inputs(1, lens, ch, N, G, dtype), lens, G, dtype)
    check(inputs(2, lens, ch, N, G, dtype, D=False, z=False, first=False, plus=False), lens, G, dtype, plus=False,
          max_len=max(lens))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,ch,N", [([700], 64, 16), ([1500, 3, 0, 400], 40, 16), ([900], 33, 5), ([640, 641], 16, 64),
                                       ([2000], 136, 8), ([769], 20, 32)])
def test_long_sequences(dtype, lens, ch, N):
    """Few channels and a long axis: sequences may be split."""
    check(inputs(3, lens, ch, N, 1, dtype), lens, 1, dtype, max_len=max(lens))
    check(inputs(4, lens, ch, N, 1, dtype), lens, 1, dtype, in_place=True)
    check(inputs(5, lens, ch, N, 1, dtype, first=False, z=False, plus=False), lens, 1, dtype, plus=False, max_len=max(lens))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 2), (8, 8), (8, 4)])
def test_strides_and_alignments(dtype, pad, offset):
    for lens in ([40, 7, 0, 90], [600]):
        check(inputs(6, lens, 40, 16, 2, dtype, pad=pad, offset=offset), lens, 2, dtype)
        check(inputs(7, lens, 33, 9, 1, dtype, pad=pad, offset=offset), lens, 1, dtype)


@pytest.mark.parametrize("lens", [[1] * 300, [2] * 130 + [400], [0] * 200 + [70]])
def test_many_sequences(lens):
    check(inputs(8, lens, 24, 16, 1, torch.bfloat16), lens, 1, torch.bfloat16)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,ch,N,G,pad,offset", [(1, 1, 1, 1, 0, 0), (3, 100, 16, 1, 0, 0), (2, 130, 16, 2, 8, 8),
                                                 (5, 66, 7, 3, 1, 1), (4, 40, 64, 1, 0, 0), (130, 24, 8, 8, 0, 0),
                                                 (9, 32, 32, 1, 3, 0), (33, 50, 12, 1, 0, 2), (2, 9, 4, 1, 0, 0)])
def test_single_tokens(dtype, n, ch, N, G, pad, offset):
    for kw in (dict(), dict(D=False, z=False, plus=False)):
        a = inputs(9, [1] * n, ch, N, G, dtype, pad=pad, offset=offset, **kw)
        plus = kw.get("plus", True)
        ref = reference(a, [1] * n, plus)
        lq.ssm_decode_step(lq.ssm_config(ch, N, G, dtype, softplus=plus), a["S0"], a["x"], a["dt"], a["A"], a["B"], a["C"],
                           a["y"], D=a["D"], z=a["z"], dt_bias=a["bias"])
        compare(a["y"], a["S0"], ref, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_parts_and_single_tokens_continue_one_another(dtype):
    T, ch, N = 90, 48, 16
    a = inputs(10, [T], ch, N, 1, dtype)
    ref = reference(a, [T], True)
    cfg, S = lq.ssm_config(ch, N, 1, dtype), a["S0"]
    part = lambda i, j: {k: v[i:j] if k in ("x", "dt", "B", "C", "y", "z") else v for k, v in a.items()}
    for i, j in ((0, 1), (1, 50), (50, 80)):
        call(cfg, part(i, j), [j - i], S)
    for t in range(80, T):
        b = part(t, t + 1)
        lq.ssm_decode_step(cfg, S, b["x"], b["dt"], b["A"], b["B"], b["C"], b["y"], D=b["D"], z=b["z"], dt_bias=b["bias"])
    compare(a["y"], S, ref, dtype)


@pytest.mark.parametrize("T", [60, 1200])
def test_steps_of_every_size(T):
    """Softplus from where it is e^v to where it is v, steps of zero, decays that are 1 and that are 0."""
    a = inputs(11, [T], 30, 16, 1, torch.float32)
    a["dt"][:] = torch.linspace(-60, 60, 30, device=DEV)
    a["bias"].zero_()
    check(a, [T], 1, torch.float32)
    a = inputs(12, [T], 30, 16, 1, torch.float32, plus=False)
    a["dt"][:, :10], a["A"][10:20] = 0.0, 0.0
    check(a, [T], 1, torch.float32, plus=False)


@pytest.mark.parametrize("T", [50, 800])
def test_growing_and_negative_steps(T):
    """A positive A and negative steps are taken as the recurrence takes them."""
    a = inputs(13, [T], 24, 8, 1, torch.float32, plus=False)
    a["A"][:8] = 0.01
    a["dt"][:, 8:16] *= -0.02
    check(a, [T], 1, torch.float32, plus=False, max_len=T)


@pytest.mark.parametrize("T", [90, 1300])
def test_values_that_are_not_finite(T):
    """They reach their own and later tokens of their channel (of every channel, from B and C), as in the recurrence."""
    a = inputs(14, [T, 40], 32, 16, 1, torch.float32)
    x, dt, z = a["x"], a["dt"], a["z"]
    x[T // 3, 2], x[T // 2, 3], x[T - 5, 4] = INF, -INF, float("nan")
    dt[T // 3, 6], dt[T // 4, 7] = INF, float("nan")
    z[T // 3, 9], z[7, 10] = INF, float("nan")
    a["S0"][0, 12, 3], a["S0"][0, 13, 5], a["S0"][1, 14, 1] = INF, float("nan"), -INF
    x[5, 16] = 3e38
    a["S0"][0, 17] = 1e38
    a["A"][18, 2], a["A"][19, 3], a["A"][20, 1] = -INF, INF, float("nan")
    a["S0"][0, 21, 0], a["A"][21, 0] = 1.0, 300.0  # grows past the largest number
    a["S0"][0, 22, 0], a["A"][22, 0] = 0.0, 300.0
    x[:, 22] = 0.0                                 # stays zero however its decays multiply
    y_r, S_r, _, _ = reference(a, [T, 40], True)
    S = torch.empty(2, 32, 16, device=DEV)
    call(lq.ssm_config(32, 16, 1, torch.float32), a, [T, 40], S, max_len=T)
    with np.errstate(over="ignore"):
        lim = float(np.finfo(np.float32).max)
        for got, want in ((f64(a["y"]), y_r), (f64(S), S_r)):
            # a sum of two infinities is NaN here where 64 bits may hold two large numbers and their difference
            sure = np.isfinite(want) & (np.abs(want) < 1e30) | np.isnan(want)
            big = np.abs(want) > 1.01 * lim
            assert np.array_equal(np.isfinite(got)[sure], np.isfinite(want)[sure])
            assert not np.isfinite(got[big]).any()
    fine = np.isfinite(S_r) & (np.abs(S_r) < 1e30)
    assert np.allclose(f64(S)[fine], S_r[fine], rtol=2e-3, atol=1e-5)


def test_bad_bounds_count_as_empty():
    cu = torch.tensor([10, 20, 5, 9, 200, 30, 95], dtype=torch.int32, device=DEV)  # 10..20, -, 5..9, -, -, 30..95 too long
    a = inputs(15, [100], 24, 16, 1, torch.float32)
    a["S0"] = torch.randn(6, 24, 16, device=DEV)
    a["y"].fill_(3.0)
    S = torch.zeros_like(a["S0"])
    cfg = lq.ssm_config(24, 16, 1, torch.float32)
    call(cfg, a, [0] * 6, S, max_len=50, cu=cu)
    for b, i, j in ((0, 10, 20), (2, 5, 9)):
        part = {k: v[i:j] if k in ("x", "dt", "B", "C", "y", "z") else v for k, v in a.items()}
        compare(part["y"], S[b:b + 1], reference(part, [j - i], True, a["S0"][b:b + 1]), torch.float32)
    for b in (1, 3, 4, 5):
        assert torch.equal(S[b], a["S0"][b])
    assert bool((a["y"][:5] == 3).all() and (a["y"][9:10] == 3).all() and (a["y"][20:] == 3).all())


def test_without_tokens_states_are_kept():
    cfg = lq.ssm_config(40, 16, 1, torch.bfloat16)
    a = inputs(16, [0, 0], 40, 16, 1, torch.bfloat16)
    S = torch.zeros_like(a["S0"])
    call(cfg, a, [0, 0], S)
    assert torch.equal(S, a["S0"])
    a["S0"] = None
    call(cfg, a, [0, 0], S)
    assert bool((S == 0).all())


@pytest.mark.parametrize("lens", [[100, 3, 0, 77], [1500]])
def test_streams_graphs_and_repeats_give_the_same_bits(lens):
    ch, N, dtype = 64, 16, torch.bfloat16
    a = inputs(17, lens, ch, N, 1, dtype)
    cfg, cu, n, T = lq.ssm_config(ch, N, 1, dtype), cu_of(lens), len(lens), sum(lens)
    S = [torch.empty_like(a["S0"]) for _ in range(3)]
    y = [torch.empty_like(a["x"]) for _ in range(3)]
    ws = [torch.empty(lq.ssm_workspace_bytes(cfg, n, T, 0), dtype=torch.uint8, device=DEV) for _ in range(3)]
    go = lambda i, **kw: lq.ssm_prefill(cfg, a["x"], a["dt"], a["A"], a["B"], a["C"], y[i], D=a["D"], z=a["z"],
                                        dt_bias=a["bias"], cu_seqlens=cu, S0=a["S0"], S_out=S[i], workspace=ws[i], **kw)
    go(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    go(1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    s, y1, torn = a["S0"].clone(), torch.empty(n, ch, dtype=dtype, device=DEV), {k: a[k][:n] for k in ("x", "dt", "B", "C", "z")}
    step = lambda s, y1: lq.ssm_decode_step(cfg, s, torn["x"], torn["dt"], a["A"], torn["B"], torn["C"], y1, D=a["D"],
                                            z=torn["z"], dt_bias=a["bias"])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream(), capture_error_mode="relaxed"):
        go(2)
        step(s, y1)
    s.copy_(a["S0"])
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for i in (1, 2):
        assert torch.equal(y[0], y[i]) and torch.equal(S[0], S[i])
    s2, y2 = a["S0"].clone(), torch.empty_like(y1)
    step(s2, y2)
    step(s2, y2)
    assert torch.equal(s, s2) and torch.equal(y1, y2)


def test_offsets_past_32_bits():
    """Tokens 2^29 elements apart: the last starts 4.3 GB in."""
    ch, N, T, stride = 40, 16, 5, 1 << 29
    a = inputs(18, [T], ch, N, 1, torch.bfloat16)
    cfg = lq.ssm_config(ch, N, 1, torch.bfloat16)
    S = torch.empty(1, ch, N, device=DEV)
    call(cfg, a, [T], S)
    want = a["y"].clone()
    for name in ("x", "z", "B", "y"):
        t = a[name]
        far = torch.empty(4 * stride + t[0].numel(), dtype=t.dtype, device=DEV).as_strided(t.shape, (stride,) + t.stride()[1:])
        far.copy_(t)
        b = dict(a, **{name: far})
        call(cfg, b, [T], S)
        assert torch.equal(b["y"], want)
        del far, b


@pytest.mark.parametrize("T,N", [(60, 5), (1300, 5), (70, 12), (50, 20)])
def test_infinities_with_any_number_of_states(T, N):
    """States are as the recurrence has them; outputs are finite exactly where it has finite ones (an infinite one may be
    NaN where n_state is not a power of two)."""
    a = inputs(19, [T], 20, N, 1, torch.float32)
    a["x"][T // 3, 2], a["x"][T - 2, 3], a["S0"][0, 7, N - 1] = INF, -INF, INF
    y_r, S_r, _, _ = reference(a, [T], True)
    S = torch.empty(1, 20, N, device=DEV)
    call(lq.ssm_config(20, N, 1, torch.float32), a, [T], S, max_len=T)
    assert np.array_equal(np.isfinite(f64(a["y"])), np.isfinite(y_r))
    got = f64(S)
    assert np.array_equal(np.isnan(got), np.isnan(S_r)) and np.array_equal(got[np.isinf(S_r)], S_r[np.isinf(S_r)])
    one, s1 = torch.empty(1, 20, device=DEV), a["S0"].clone()
    t = T // 3
    part = {k: v[t:t + 1] if k in ("x", "dt", "B", "C", "y", "z") else v for k, v in a.items()}
    y1, S1, _, _ = reference(part, [1], True, s1)
    lq.ssm_decode_step(lq.ssm_config(20, N, 1, torch.float32), s1, part["x"], part["dt"], a["A"], part["B"], part["C"], one,
                       D=a["D"], z=part["z"], dt_bias=a["bias"])
    assert np.array_equal(np.isfinite(f64(one)), np.isfinite(y1))
    assert np.array_equal(f64(s1)[np.isinf(S1)], S1[np.isinf(S1)]) and not np.isnan(f64(s1)).any()
