"""Linear attention with a decay per head (lq_la_prefill, lq_la_decode_step) against the 64-bit recurrence."""
import numpy as np
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests._generation import D, la_reference, output_bound, rel, state_bound

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


def inputs(seed, lens, heads, key_heads, dtype, first=False, fused=False, half_life=(1.0, 3000.0)):
    rng = np.random.default_rng(seed)
    T, B = sum(lens), len(lens)
    lo, hi = half_life
    alpha = np.exp2(-1.0 / np.exp(rng.uniform(np.log(lo), np.log(hi), (T, heads)))).astype(np.float32)
    if fused:
        rows = torch.from_numpy(rng.standard_normal((T, (2 * key_heads + heads) * D)).astype(np.float32))
        rows[:, key_heads * D:2 * key_heads * D] *= D ** -0.5
        rows = rows.to(DEV, dtype)
        q, k, v = (x.view(T, -1, D) for x in rows.split([key_heads * D, key_heads * D, heads * D], dim=1))
    else:
        mk = lambda n, s: torch.from_numpy((rng.standard_normal((T, n, D)) * s).astype(np.float32)).to(DEV, dtype)
        q, k, v = mk(key_heads, 1.0), mk(key_heads, D ** -0.5), mk(heads, 1.0)
    S0 = torch.from_numpy((0.3 * rng.standard_normal((B, heads, D, D))).astype(np.float32)).to(DEV) if first else None
    return q, k, v, torch.from_numpy(alpha).to(DEV), S0


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)


def workspace(cfg, n_seqs, n_tokens, max_len):
    n = lq.la_workspace_bytes(cfg, n_seqs, n_tokens, max_len)
    return torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None  # NaN, should anything read it first


def run(q, k, v, alpha, lens, S0=None, known=True, cu="make", S_out=True, stream=None):
    H, K, T, B = v.shape[1], k.shape[1], v.shape[0], len(lens)
    cfg = lq.la_config(H, K, q.dtype)
    o = torch.full((T, H, D), 77.0, dtype=q.dtype, device=DEV)
    S = torch.full((B, H, D, D), 77.0, device=DEV) if S_out is True else S_out
    max_len = max(lens) if known else 0
    lq.la_prefill(cfg, q, k, v, alpha, o, cu_seqlens=cu_of(lens) if isinstance(cu, str) else cu, max_len=max_len,
                  S0=S0, S_out=S, workspace=workspace(cfg, B, T, max_len), stream=stream)
    return o, S


def f64(x):
    return x.double().cpu().numpy()


def check(q, k, v, alpha, lens, S0, o, S):
    o_r, S_r = la_reference(f64(q), f64(k), f64(v), f64(alpha), lens, None if S0 is None else f64(S0))
    n = max(lens)
    assert rel(f64(o), o_r) <= output_bound(q.dtype, n), rel(f64(o), o_r)
    if S is not None:
        assert rel(f64(S), S_r) <= state_bound(n), rel(f64(S), S_r)
        for b in range(len(lens)):  # no sequence hides behind the others
            assert rel(f64(S[b]), S_r[b]) <= 2 * state_bound(n)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", [[1], [2], [17], [64], [63, 64, 65], [127, 128, 129, 1], [0, 5, 0, 200, 3, 0]])
def test_lengths(dtype, lens):
    q, k, v, a, S0 = inputs(len(lens), lens, 2, 2, dtype, first=len(lens) % 2 == 0)
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,key_heads", [(1, 1), (3, 1), (6, 2), (8, 8)])
@pytest.mark.parametrize("fused", [False, True])
def test_head_layouts(dtype, heads, key_heads, fused):
    lens = [70, 150]
    q, k, v, a, S0 = inputs(heads * 10 + key_heads, lens, heads, key_heads, dtype, first=True, fused=fused)
    o, S = run(q, k, v, a, lens, S0, known=not fused)
    check(q, k, v, a, lens, S0, o, S)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("known", [False, True])
def test_long_sequences_are_split(dtype, known):
    lens = [3001, 64, 2500] if known else [2900]
    q, k, v, a, S0 = inputs(5, lens, 1, 1, dtype, first=known, half_life=(20.0, 20000.0))
    o, S = run(q, k, v, a, lens, S0, known=known)
    check(q, k, v, a, lens, S0, o, S)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["ones", "zeros", "some zeros", "tiny", "negative", "above one", "fixed"])
def test_decays(dtype, kind):
    lens = [200, 90]
    q, k, v, a, S0 = inputs(6, lens, 2, 1, dtype, first=True)
    if kind == "ones":
        a.fill_(1.0)
    elif kind == "zeros":
        a.zero_()
    elif kind == "some zeros":
        a[::37] = 0.0
    elif kind == "tiny":
        a.mul_(1e-30)
    elif kind == "negative":
        a[::3] *= -1.0
    elif kind == "above one":
        a.fill_(1.003)
    elif kind == "fixed":
        a = a[7:8].expand(290, 2)
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)


@pytest.mark.parametrize("dtype", TYPES)
def test_fast_decays_keep_their_accuracy(dtype):
    """Half-lives of a twentieth of a token: every weight is the product of few decays, though the logarithms'
    sums over a chunk are in the thousands."""
    lens = [400]
    q, k, v, a, S0 = inputs(7, lens, 2, 2, dtype, half_life=(0.05, 0.3))
    o, S = run(q, k, v, a, lens, S0)
    check(q, k, v, a, lens, S0, o, S)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("what", ["v", "k", "q"])
def test_infinities_and_nan_reach_later_tokens_only(dtype, value, what):
    lens = [150, 140, 64]
    q, k, v, a, S0 = inputs(8, lens, 2, 2, dtype)
    clean_o, clean_S = run(q, k, v, a, lens, S0)
    at = 150 + 77
    {"v": v, "k": k, "q": q}[what][at, 1, 5] = value
    o, S = run(q, k, v, a, lens, S0)
    o_r, S_r = la_reference(f64(q), f64(k), f64(v), f64(a), lens)
    got, want = f64(o), o_r
    same = np.ones(o.shape, bool)
    same[150:290, 1] = False
    assert np.array_equal(got[same], f64(clean_o)[same])
    assert np.array_equal(np.isfinite(got), np.isfinite(want))
    assert np.array_equal(np.isfinite(f64(S)), np.isfinite(S_r))
    fine = np.isfinite(want)
    assert rel(got[fine], want[fine]) <= output_bound(dtype, 150)
    fine = np.isfinite(S_r)
    assert rel(f64(S)[fine], S_r[fine]) <= state_bound(150)
    assert torch.equal(S[0], clean_S[0]) and torch.equal(S[2], clean_S[2])


@pytest.mark.parametrize("dtype", TYPES)
def test_extreme_magnitudes(dtype):
    """Values near the type's largest and far below one keep the relative accuracy of their own scale."""
    lens = [130]
    q, k, v, a, _ = inputs(9, lens, 2, 1, dtype)
    big = {torch.float16: 2e4, torch.bfloat16: 1e30, torch.float32: 1e30}[dtype]
    v[:, 0] *= big / 8
    v[:, 1] *= 2.0 ** -12
    o = run(q, k, v, a, lens, S_out=True)
    o_r, S_r = la_reference(f64(q), f64(k), f64(v), f64(a), lens)
    for h in range(2):
        assert rel(f64(o[1][:, h]), S_r[:, h]) <= state_bound(130)
        fits = np.abs(o_r[:, h]) < 0.9 * torch.finfo(dtype).max
        if h == 1 and dtype == torch.float16:  # below fp16's normal numbers the outputs' own steps are absolute
            assert np.abs(f64(o[0][:, h]) - o_r[:, h]).max() <= output_bound(dtype, 130) * np.abs(o_r[:, h]).max()
        else:
            assert rel(f64(o[0][:, h])[fits], o_r[:, h][fits]) <= output_bound(dtype, 130)


def test_bad_bounds_count_as_empty():
    """Bounds that decrease, run past the tokens, are negative or exceed a stated max_len read and write nothing."""
    lens = [40, 30, 50]
    q, k, v, a, S0 = inputs(10, lens, 2, 2, torch.bfloat16, first=True)
    o_good, S_good = run(q, k, v, a, lens, S0)
    for bad, empty in [([0, 40, 30, 120], [1]), ([0, 40, 70, 121], [2]), ([-5, 40, 70, 120], [0]),
                       ([0, 40, 2**31 - 1, 120], [1, 2])]:
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        cfg = lq.la_config(2, 2, torch.bfloat16)
        o = torch.full_like(o_good, 77.0)
        S = torch.full_like(S_good, 77.0)
        lq.la_prefill(cfg, q, k, v, a, o, cu_seqlens=cu, S0=S0, S_out=S, workspace=workspace(cfg, 3, 120, 0))
        for b in range(3):
            if b in empty:
                assert torch.equal(S[b], S0[b]), (bad, b)
        if 0 not in empty:
            assert torch.equal(S[0], S_good[0]) and torch.equal(o[:30], o_good[:30])
        if bad == [0, 40, 70, 121]:
            assert bool((o[70:] == 77.0).all())


def test_in_place_states_and_no_last_states():
    lens = [90, 300]
    q, k, v, a, S0 = inputs(11, lens, 4, 2, torch.bfloat16, first=True)
    o1, S1 = run(q, k, v, a, lens, S0)
    S = S0.clone()
    o2, _ = run(q, k, v, a, lens, S, S_out=S)
    assert torch.equal(S, S1) and torch.equal(o1, o2)
    o3, none = run(q, k, v, a, lens, S0, S_out=None)
    assert none is None and torch.equal(o1, o3)


def test_one_sequence_needs_no_bounds_and_no_tokens_are_fine():
    q, k, v, a, S0 = inputs(12, [77], 2, 2, torch.float32, first=True)
    o1, S1 = run(q, k, v, a, [77], S0)
    o2, S2 = run(q, k, v, a, [77], S0, cu=None)
    assert torch.equal(o1, o2) and torch.equal(S1, S2)
    _, S3 = run(q[:0], k[:0], v[:0], a[:0], [0], S0, cu=None, known=False)
    assert torch.equal(S3, S0)
    _, S4 = run(q[:0], k[:0], v[:0], a[:0], [0, 0], None, known=False)
    assert bool((S4 == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_parts_of_a_prompt_and_single_tokens_continue_each_other(dtype):
    """200 tokens at once, or 120 and 79 and the last one by the recurrent form."""
    lens = [200]
    q, k, v, a, S0 = inputs(13, lens, 4, 2, dtype, first=True)
    o, S = run(q, k, v, a, lens, S0)
    x = S0.clone()
    parts = []
    for t0, t1 in ((0, 120), (120, 199)):
        y, _ = run(q[t0:t1], k[t0:t1], v[t0:t1], a[t0:t1], [t1 - t0], x, S_out=x)
        parts.append(y)
    last = torch.empty(1, 4, D, dtype=dtype, device=DEV)
    lq.la_decode_step(lq.la_config(4, 2, dtype), x, q[199:], k[199:], v[199:], a[199:], last)
    got = torch.cat(parts + [last])
    check(q, k, v, a, lens, S0, got, x)
    assert rel(f64(got), f64(o)) <= 2 * output_bound(dtype, 200)


def test_streams_graphs_and_repeats_give_the_same_bits():
    lens = [700, 30]
    q, k, v, a, S0 = inputs(14, lens, 2, 2, torch.bfloat16, first=True)
    o1, S1 = run(q, k, v, a, lens, S0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, S2 = run(q, k, v, a, lens, S0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o1, o2) and torch.equal(S1, S2)
    cfg, cu = lq.la_config(2, 2), cu_of(lens)
    ws = workspace(cfg, 2, 730, 700)
    o3, S3 = torch.zeros_like(o1), torch.zeros_like(S1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream(), capture_error_mode="relaxed"):
        lq.la_prefill(cfg, q, k, v, a, o3, cu_seqlens=cu, max_len=700, S0=S0, S_out=S3, workspace=ws)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, o3) and torch.equal(S1, S3)


def test_token_offsets_past_32_bits():
    """Tokens 2^18 elements apart: the last of 9,000 starts 4.7 GB into its array."""
    T, stride = 9000, 1 << 18
    q, k, v, a, _ = inputs(15, [T], 1, 1, torch.bfloat16)
    flat = torch.zeros(T * stride, dtype=torch.bfloat16, device=DEV)
    wide = flat.view(T, 1, stride)
    parts = []
    for i, x in enumerate((q, k, v)):
        part = wide[:, :, i * D:(i + 1) * D]
        part.copy_(x)
        parts.append(part)
    o1, S1 = run(q, k, v, a, [T])
    cfg = lq.la_config(1, 1)
    o2 = torch.empty(T * stride, dtype=torch.bfloat16, device=DEV).view(T, 1, stride)[:, :, :D]
    S2 = torch.empty_like(S1)
    lq.la_prefill(cfg, *parts, a, o2, max_len=T, S_out=S2, workspace=workspace(cfg, 1, T, T))
    assert torch.equal(o1, o2) and torch.equal(S1, S2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,heads,key_heads", [(1, 1, 1), (1, 3, 1), (5, 6, 2), (40, 16, 16)])
def test_single_tokens(dtype, n, heads, key_heads):
    q, k, v, a, S0 = inputs(n, [1] * n, heads, key_heads, dtype, first=True, fused=n == 5)
    S = S0.clone()
    o = torch.empty(n, heads, D, dtype=dtype, device=DEV)
    lq.la_decode_step(lq.la_config(heads, key_heads, dtype), S, q, k, v, a, o)
    check(q, k, v, a, [1] * n, S0, o, S)


def test_single_tokens_of_any_value():
    q, k, v, a, S0 = inputs(3, [1] * 4, 2, 2, torch.float32, first=True)
    a[0, 0], a[1, 0], a[2, 0] = 0.0, -0.5, float("nan")
    v[3, 1, 9] = float("inf")
    S = S0.clone()
    o = torch.empty(4, 2, D, device=DEV)
    lq.la_decode_step(lq.la_config(2, 2, torch.float32), S, q, k, v, a, o)
    o_r, S_r = la_reference(f64(q), f64(k), f64(v), f64(a), [1] * 4, f64(S0))
    assert np.array_equal(np.isfinite(f64(S)), np.isfinite(S_r))
    assert np.array_equal(np.isfinite(f64(o)), np.isfinite(o_r))
    fine = np.isfinite(S_r)
    assert rel(f64(S)[fine], S_r[fine]) <= state_bound(1)


def test_states_go_on_into_the_quantized_decode():
    """A prompt's last states are what lq_state_init_range takes: exported at once they come back within the
    8-bit boundary's error, row by row at most half a step."""
    q, k, v, a, _ = inputs(16, [300, 200], 4, 4, torch.bfloat16)
    _, S = run(q, k, v, a, [300, 200])
    cfg = lq.config(n_comp=0, smooth=False)
    state = lq.alloc_state(cfg, 8, DEV)
    lq.state_init(cfg, state, 8, None)
    lq.state_init_range(cfg, state, 8, 4, 4, S[1])
    back = torch.empty(8, D, D, device=DEV)
    lq.export_state(cfg, state, 8, back)
    assert lq.get_status(state)[0] == lq.OK
    off = (back[4:] - S[1].view(4, D, D)).abs().amax(-1)
    assert bool((off <= S[1].view(4, D, D).abs().amax(-1) / 127 * (0.5 + 1e-5)).all())
