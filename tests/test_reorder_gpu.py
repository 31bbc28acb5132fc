"""Head-states that follow the hypotheses chosen (lq_state_reorder, lq_fp32_state_reorder): exact copies."""
import numpy as np
import pytest
import torch

from quantized_linear_attention_gb300 import lq
from tests._generation import D, reorder_reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lq.load()
    torch.cuda.set_device(0)


def filled(cfg, n, seed):
    """A state buffer with arbitrary plane contents and record counts."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    state = torch.zeros(lq.state_bytes(cfg, n), dtype=torch.uint8, device=DEV)
    lq.state_init(cfg, state, n, None)
    views = lq.state_views(cfg, state, n)
    for name, x in views.items():
        if name == "counts":
            x.copy_(torch.randint(0, cfg.window + 1, x.shape, generator=g, device=DEV))
        elif name == "full_list":
            continue
        elif x.dtype == torch.float32:
            x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        else:
            x.copy_(torch.randint(0, 120, x.shape, generator=g, device=DEV).to(x.dtype))
    return state, views


def arrays(views):
    return {k: x.cpu().numpy().copy() for k, x in views.items()}


def parents(seed, groups, beams):
    return np.random.default_rng(seed).integers(0, beams, (groups, beams)).astype(np.int32)


CONFIGS = [dict(), dict(kda=True), dict(code_bits=4, n_comp=0), dict(code_bits=6, n_comp=3, window=5),
           dict(comp_fit=2, n_comp=2, window=32), dict(kda=True, window=1, n_comp=8)]


@pytest.mark.parametrize("kw", CONFIGS)
@pytest.mark.parametrize("outer,groups,beams,inner", [(1, 1, 1, 1), (2, 3, 4, 5), (1, 2, 7, 3), (3, 1, 16, 2),
                                                      (1, 2, 32, 1)])
def test_quantized_states(kw, outer, groups, beams, inner):
    cfg = lq.config(**kw)
    n = outer * groups * beams * inner
    state, views = filled(cfg, n, beams)
    before = arrays(views)
    par = parents(beams + inner, groups, beams)
    want = reorder_reference(before, par, outer, inner, counts=before["counts"])
    lq.state_reorder(cfg, state, n, torch.from_numpy(par).to(DEV), outer=outer, inner=inner)
    assert lq.get_status(state) == (lq.OK, -1)
    got = arrays(views)
    for name in before:
        assert np.array_equal(got[name], want[name], equal_nan=True), name


@pytest.mark.parametrize("perm", ["identity", "reverse", "rotate", "fork", "swap"])
def test_parents(perm):
    K = 6
    par = {"identity": list(range(K)), "reverse": list(range(K))[::-1], "rotate": [1, 2, 3, 4, 5, 0], "fork": [0] * K,
           "swap": [1, 0, 2, 3, 5, 4]}[perm]
    S = torch.randn(2, 2, K, 3, D, D, device=DEV)  # outer 2, groups 2, inner 3
    want = S[:, :, par].clone()
    lq.fp32_state_reorder(S, torch.tensor([par, par], dtype=torch.int32, device=DEV), outer=2, inner=3)
    assert torch.equal(S, want)


@pytest.mark.parametrize("beams", [1, 3, 4, 5, 8, 9, 16, 17, 32])
def test_fp32_states(beams):
    S = torch.randn(3, beams, 2, D, D, device=DEV)
    par = parents(beams, 3, beams)
    want = torch.stack([S[g][par[g].tolist()] for g in range(3)])
    lq.fp32_state_reorder(S, torch.from_numpy(par).to(DEV), inner=2)
    assert torch.equal(S, want)


def test_a_bad_parent_leaves_its_group_and_says_so():
    cfg = lq.config(window=4)
    n = 2 * 3 * 4 * 2
    state, views = filled(cfg, n, 1)
    before = arrays(views)
    par = parents(2, 3, 4)
    for bad in (4, -1, 2**31 - 1):
        par[1] = [0, bad, 1, 1]
        want = reorder_reference(arrays(views), par, 2, 2, counts=arrays(views)["counts"])
        lq.state_reorder(cfg, state, n, torch.from_numpy(par).to(DEV), outer=2, inner=2)
        status, at = lq.get_status(state)
        assert status == lq.ERR_PARENT and (at // 8) % 3 == 1
        got = arrays(views)
        for name in before:
            assert np.array_equal(got[name], want[name]), name
        lq.clear_status(state)
    S = torch.randn(3, 4, D, D, device=DEV)
    want = torch.stack([S[0][par[0].tolist()], S[1], S[2][par[2].tolist()]])
    lq.fp32_state_reorder(S, torch.from_numpy(par).to(DEV))
    assert torch.equal(S, want)


def test_bad_counts_and_buffers_are_left():
    cfg = lq.config()
    state, views = filled(cfg, 8, 3)
    views["counts"][5] = 17
    before = arrays(views)
    par = torch.tensor([[1, 0, 3, 2], [1, 0, 3, 2]], dtype=torch.int32, device=DEV)
    lq.state_reorder(cfg, state, 8, par)
    assert lq.get_status(state)[0] == lq.ERR_STATE
    got = arrays(views)
    assert np.array_equal(got["codes"][4:], before["codes"][4:])
    assert np.array_equal(got["codes"][:4], before["codes"][[1, 0, 3, 2]])
    other = lq.config(window=8)
    lq.clear_status(state)
    whole = state.clone()
    lq.state_reorder(other, state, 8, par)
    assert lq.get_status(state)[0] == lq.ERR_STATE
    assert torch.equal(whole[256:], state[256:])


def test_decoding_goes_on_after_a_reordering():
    """Beams that took over another one's state decode as that one does, through the window's fold."""
    K, cfg = 4, lq.config(window=4, n_comp=2)
    g = torch.Generator(device=DEV).manual_seed(4)
    S0 = torch.randn(K, D, D, generator=g, device=DEV) * 0.1
    par = torch.tensor([[2, 2, 0, 3]], dtype=torch.int32, device=DEV)
    tok = [[torch.randn(K, D, generator=g, device=DEV) for _ in range(3)] for _ in range(7)]
    a, b = torch.full((K,), 0.97, device=DEV), torch.full((K,), 0.5, device=DEV)
    state, o = lq.alloc_state(cfg, K), torch.empty(K, D, device=DEV)
    lq.state_init(cfg, state, K, S0)
    direct, o2 = lq.alloc_state(cfg, K), torch.empty(K, D, device=DEV)
    src = par[0].long()
    lq.state_init(cfg, direct, K, S0[src].contiguous())
    for t, (q, k, v) in enumerate(tok):
        k = k / k.norm(dim=1, keepdim=True)
        if t == 3:
            lq.state_reorder(cfg, state, K, par)
        if t < 3:
            lq.decode_step(cfg, state, K, q, k, v, a, b, o)
            lq.decode_step(cfg, direct, K, q[src].contiguous(), k[src].contiguous(), v[src].contiguous(), a, b, o2)
        else:
            lq.decode_step(cfg, state, K, q, k, v, a, b, o)
            lq.decode_step(cfg, direct, K, q, k, v, a, b, o2)
            assert torch.equal(o, o2)
    assert lq.get_status(state)[0] == lq.OK
    x, y = torch.empty(K, D, D, device=DEV), torch.empty(K, D, D, device=DEV)
    lq.export_state(cfg, state, K, x)
    lq.export_state(cfg, direct, K, y)
    assert torch.equal(x, y)


def test_offsets_past_32_bits_and_graphs():
    """70,000 fp32 states: 4.6 GB, the last group's beams exchanged."""
    n = 70000
    S = torch.zeros(n, D, D, device=DEV)
    S[-2:] = torch.randn(2, D, D, device=DEV)
    want = S[-2:].flip(0).clone()
    par = torch.tensor([[0, 1]], dtype=torch.int32, device=DEV).repeat(n // 2, 1)
    par[-1] = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream(), capture_error_mode="relaxed"):
        lq.fp32_state_reorder(S, par)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(S[-2:], want) and not bool(S[:-2].any())
