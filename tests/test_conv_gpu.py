"""The short causal convolution (lq_conv_prefill, lq_conv_decode_step) against its definition in 64 bits."""
import numpy as np
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests._layers import conv_bound, conv_reference

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
    T, C = t.shape
    flat = torch.full((T * (C + pad) + offset,), fill, dtype=t.dtype, device=DEV)
    v = flat[offset:].view(T, C + pad)[:, :C]
    v.copy_(t)
    return v


def inputs(seed, lens, C, W, dtype, bias=True, first=True, pad=0, offset=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    T, B = sum(lens), len(lens)
    return dict(x=rows(r(T, C).to(dtype), pad, offset), weight=r(C, W), bias=r(C) if bias else None,
                S0=r(B, W - 1, C).to(dtype) if first else None, y=rows(torch.zeros(T, C, dtype=dtype, device=DEV), pad, offset, 5.0))


def check(a, lens, W, act, dtype, max_len=0, in_place=False, cu=True):
    C = a["x"].shape[1]
    y_r, S_r, mag = conv_reference(f64(a["x"]), f64(a["weight"]), f64(a["bias"]), lens, f64(a["S0"]), act)
    S = a["S0"] if in_place else torch.full((len(lens), W - 1, C), 7.0, dtype=dtype, device=DEV)
    cfg = lq.conv_config(C, W, dtype, silu=act)
    lq.conv_prefill(cfg, a["x"], a["weight"], a["y"], bias=a["bias"], cu_seqlens=cu_of(lens) if cu else None,
                    max_len=max_len, S0=a["S0"], S_out=S)
    y = f64(a["y"])
    assert np.all(np.abs(y - y_r) <= conv_bound(y_r, mag, dtype)), np.abs(y - y_r).max()
    assert np.array_equal(f64(S), S_r)
    return S


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens,C", [([1], 1), ([2], 8), ([3], 129), ([5, 0, 1, 2, 33, 32, 31], 64), ([200], 1027),
                                    ([64, 1, 65], 2048), ([300, 17], 256)])
def test_lengths_and_channels(dtype, W, lens, C):
    check(inputs(1, lens, C, W, dtype), lens, W, True, dtype)
    check(inputs(2, lens, C, W, dtype, bias=False, first=False), lens, W, False, dtype, max_len=max(lens))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,offset", [(0, 1), (8, 0), (1, 0), (3, 2), (8, 8), (8, 4)])
def test_strides_and_alignments(dtype, pad, offset):
    lens = [40, 7, 0, 90]
    check(inputs(3, lens, 520, 4, dtype, pad=pad, offset=offset), lens, 4, True, dtype)


@pytest.mark.parametrize("dtype", TYPES)
def test_state_in_place(dtype):
    for lens in ([1], [2, 3, 100, 0], [4, 1, 1]):
        check(inputs(4, lens, 72, 4, dtype), lens, 4, True, dtype, in_place=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,C", [([1] * 1000, 136), ([3] * 300 + [500], 40), ([0] * 257 + [65], 16)])
def test_many_sequences(dtype, lens, C):
    check(inputs(5, lens, C, 4, dtype), lens, 4, True, dtype)


def test_one_sequence_without_bounds():
    check(inputs(6, [333], 96, 3, torch.bfloat16), [333], 3, True, torch.bfloat16, cu=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_prompts_in_parts_and_single_tokens_are_the_whole(dtype):
    """One prompt, the same in three parts, the same token by token: the same values in the same order, the same bits."""
    T, C, W = 50, 200, 4
    a = inputs(7, [T], C, W, dtype)
    cfg = lq.conv_config(C, W, dtype)
    S = torch.empty(1, W - 1, C, dtype=dtype, device=DEV)
    lq.conv_prefill(cfg, a["x"], a["weight"], a["y"], bias=a["bias"], S0=a["S0"], S_out=S)
    parts, s1 = torch.zeros_like(a["y"]), a["S0"].clone()
    for i, j in ((0, 2), (2, 37), (37, 50)):
        lq.conv_prefill(cfg, a["x"][i:j], a["weight"], parts[i:j], bias=a["bias"], S0=s1, S_out=s1)
    single, s2 = torch.zeros_like(a["y"]), a["S0"].clone()
    for t in range(T):
        lq.conv_decode_step(cfg, s2, a["x"][t:t + 1], a["weight"], single[t:t + 1], bias=a["bias"])
    for y, s in ((parts, s1), (single, s2)):
        assert torch.equal(y, a["y"]) and torch.equal(s, S)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("n,C,pad,offset", [(1, 1, 0, 0), (3, 515, 0, 0), (7, 1024, 8, 0), (2, 64, 1, 3), (130, 24, 0, 0),
                                            (515, 264, 8, 8)])
def test_single_tokens(dtype, W, n, C, pad, offset):
    a = inputs(8, [1] * n, C, W, dtype, pad=pad, offset=offset)
    y_r, S_r, mag = conv_reference(f64(a["x"]), f64(a["weight"]), f64(a["bias"]), [1] * n, f64(a["S0"]), True)
    lq.conv_decode_step(lq.conv_config(C, W, dtype), a["S0"], a["x"], a["weight"], a["y"], bias=a["bias"])
    y = f64(a["y"])
    assert np.all(np.abs(y - y_r) <= conv_bound(y_r, mag, dtype)) and np.array_equal(f64(a["S0"]), S_r)


def test_bad_bounds_count_as_empty():
    """Sequences with bounds outside the tokens, backwards or longer than stated keep their states; others are served;
    tokens of no sequence keep what y held."""
    cu = torch.tensor([10, 20, 5, 9, 200, 30, 95], dtype=torch.int32, device=DEV)  # 10..20, -, 5..9, -, -, 30..95 too long
    a = inputs(9, [100], 48, 4, torch.float32, first=False)
    g = torch.Generator(device=DEV).manual_seed(1)
    S0 = torch.randn(6, 3, 48, generator=g, device=DEV)
    S = torch.zeros_like(S0)
    a["y"].fill_(3.0)
    lq.conv_prefill(lq.conv_config(48, 4, torch.float32), a["x"], a["weight"], a["y"], bias=a["bias"], cu_seqlens=cu,
                    max_len=50, S0=S0, S_out=S)
    for b, i, j in ((0, 10, 20), (2, 5, 9)):
        y_r, S_r, mag = conv_reference(f64(a["x"][i:j]), f64(a["weight"]), f64(a["bias"]), [j - i], f64(S0[b:b + 1]), True)
        assert np.all(np.abs(f64(a["y"][i:j]) - y_r) <= conv_bound(y_r, mag, torch.float32))
        assert np.array_equal(f64(S[b:b + 1]), S_r)
    for b in (1, 3, 4, 5):
        assert torch.equal(S[b], S0[b])
    assert bool((a["y"][:5] == 3).all() and (a["y"][9:10] == 3).all() and (a["y"][20:] == 3).all())


def test_infinities_and_nans_stay_in_their_channel_and_reach():
    a = inputs(10, [40], 16, 4, torch.float32, first=False)
    a["x"][10, 3], a["x"][20, 5], a["x"][30, 7] = INF, float("nan"), -INF
    lq.conv_prefill(lq.conv_config(16, 4, torch.float32, silu=False), a["x"], a["weight"], a["y"], bias=a["bias"])
    bad = ~torch.isfinite(a["y"])
    want = torch.zeros_like(bad)
    for t, c in ((10, 3), (20, 5), (30, 7)):
        want[t:t + 4, c] = True
    assert torch.equal(bad, want)


def test_streams_graphs_and_repeats_give_the_same_bits():
    lens, W, C, dtype = [100, 3, 0, 77], 4, 640, torch.bfloat16
    a = inputs(11, lens, C, W, dtype)
    cfg, cu = lq.conv_config(C, W, dtype), cu_of(lens)
    S = [torch.empty_like(a["S0"]) for _ in range(3)]
    y = [torch.empty_like(a["x"]) for _ in range(3)]
    call = lambda i, **kw: lq.conv_prefill(cfg, a["x"], a["weight"], y[i], bias=a["bias"], cu_seqlens=cu, S0=a["S0"], S_out=S[i], **kw)
    call(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    step, s, x1 = torch.empty(4, C, dtype=dtype, device=DEV), a["S0"].clone(), a["x"][:4]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream(), capture_error_mode="relaxed"):
        call(2)
        lq.conv_decode_step(cfg, s, x1, a["weight"], step, bias=a["bias"])
    s.copy_(a["S0"])
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for i in (1, 2):
        assert torch.equal(y[0], y[i]) and torch.equal(S[0], S[i])
    s2, step2 = a["S0"].clone(), torch.empty_like(step)
    for _ in range(2):
        lq.conv_decode_step(cfg, s2, x1, a["weight"], step2, bias=a["bias"])
    assert torch.equal(s, s2) and torch.equal(step, step2)


def test_offsets_past_32_bits():
    """Tokens 2^29 elements apart: the last starts 8.6 GB in."""
    C, stride, T = 136, 1 << 29, 9
    a = inputs(12, [T], C, 4, torch.bfloat16)
    far = torch.empty(8 * stride + C, dtype=torch.bfloat16, device=DEV).as_strided((T, C), (stride, 1))
    far.copy_(a["x"])
    cfg = lq.conv_config(C, 4, torch.bfloat16)
    want = torch.empty(T, C, dtype=torch.bfloat16, device=DEV)
    lq.conv_prefill(cfg, a["x"], a["weight"], want, bias=a["bias"])
    lq.conv_prefill(cfg, far, a["weight"], a["y"], bias=a["bias"])
    assert torch.equal(a["y"], want)
    lq.conv_prefill(cfg, a["x"], a["weight"], far, bias=a["bias"])
    assert torch.equal(far, want)


def test_without_tokens_states_are_kept():
    cfg = lq.conv_config(24, 4, torch.bfloat16)
    a = inputs(13, [0, 0], 24, 4, torch.bfloat16)
    S = torch.zeros_like(a["S0"])
    lq.conv_prefill(cfg, a["x"], a["weight"], a["y"], cu_seqlens=cu_of([0, 0]), S0=a["S0"], S_out=S)
    assert torch.equal(S, a["S0"])
    lq.conv_prefill(cfg, a["x"], a["weight"], a["y"], cu_seqlens=cu_of([0, 0]), S_out=S)
    assert bool((S == 0).all())
    lq.conv_decode_step(cfg, S[:0], a["x"], a["weight"], a["y"])
