"""What the generation calls refuse, on the host (no GPU): the checks that need no device come first, so
addresses stand in for buffers."""
import ctypes

import numpy as np
import pytest

from quantized_linear_attention_gb300 import build as lq_build
from quantized_linear_attention_gb300 import lq
from tests._generation import beam_reference, la_reference, reorder_reference

GB = 1 << 30
Q, K, V, A, O, S0, S, WS, CU = ((i + 1) * 16 * GB for i in range(9))


@pytest.fixture(scope="module")
def L():
    lq_build.build_lq()
    return lq.load()


def config(L, heads=4, key_heads=2, dtype=lq.BF16, **kw):
    c = lq.LaConfig()
    L.lq_la_config_default(ctypes.byref(c), heads, key_heads, dtype)
    for name, x in kw.items():
        setattr(c, name, x)
    return c


def prefill(L, c, n_seqs=2, n_tokens=100, max_len=0, cu=CU, q=Q, k=K, v=V, a=A, s0=S0, s=S, o=O, ws=WS, nbytes=1 << 40):
    return L.lq_la_prefill(ctypes.byref(c) if c is not None else None, n_seqs, n_tokens, max_len, cu, q, k, v, a, s0, s,
                           o, ws, nbytes, None)


def step(L, c, n=3, s=S, q=Q, k=K, v=V, a=A, o=O):
    return L.lq_la_decode_step(ctypes.byref(c), s, n, q, k, v, a, o, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d_k=64), lq.ERR_UNSUPPORTED), (dict(d_v=256), lq.ERR_UNSUPPORTED), (dict(dtype=3), lq.ERR_INVALID_ARG),
    (dict(dtype=-1), lq.ERR_INVALID_ARG), (dict(heads=5), lq.ERR_INVALID_ARG), (dict(heads=0), lq.ERR_INVALID_ARG),
    (dict(key_heads=0), lq.ERR_INVALID_ARG), (dict(reserved=1), lq.ERR_INVALID_ARG),
    (dict(q_stride=128), lq.ERR_INVALID_ARG), (dict(k_stride=257), lq.ERR_INVALID_ARG),
    (dict(v_stride=516), lq.ERR_INVALID_ARG), (dict(o_stride=-512), lq.ERR_INVALID_ARG),
    (dict(alpha_stride=3), lq.ERR_INVALID_ARG), (dict(q_stride=2**41), lq.ERR_INVALID_ARG)])
def test_configurations_refused(L, kw, code):
    c = config(L, **kw)
    assert prefill(L, c) == code and step(L, c) == code
    assert lq.last_error() != ""
    assert L.lq_la_workspace_bytes(ctypes.byref(c), 2, 100, 0) == 0


def test_prompt_arguments_refused(L):
    c = config(L)
    bad = lq.ERR_INVALID_ARG
    assert prefill(L, None) == bad
    assert prefill(L, c, n_seqs=0) == lq.OK  # nothing to do
    for kw in (dict(n_seqs=-1), dict(n_tokens=-1), dict(max_len=-1), dict(n_tokens=2**31), dict(n_seqs=2**31),
               dict(cu=None), dict(q=None), dict(k=None), dict(v=None), dict(a=None), dict(o=None), dict(q=Q + 8),
               dict(k=K + 2), dict(v=V + 4), dict(a=A + 2), dict(o=O + 8), dict(s0=S0 + 8), dict(s=S + 4),
               dict(cu=CU + 2), dict(cu=None, n_seqs=1, max_len=50), dict(o=Q + 4096), dict(o=V), dict(o=A),
               dict(s=S0 + 4096), dict(s=Q), dict(s=O), dict(s0=O), dict(s=V + 256)):
        assert prefill(L, c, **kw) == bad, kw
        assert lq.last_error() != "", kw


def test_split_prompts_need_their_workspace(L):
    c = config(L, heads=1, key_heads=1)
    need = L.lq_la_workspace_bytes(ctypes.byref(c), 1, 100000, 100000)
    if not need:
        pytest.skip("no sequence is split")
    args = dict(n_seqs=1, n_tokens=100000, max_len=100000, cu=None)
    for kw in (dict(ws=None), dict(ws=WS + 16), dict(nbytes=need - 1), dict(ws=O), dict(ws=S), dict(ws=S0), dict(ws=Q)):
        assert prefill(L, c, **args, **kw) == lq.ERR_INVALID_ARG, kw
        assert "workspace" in lq.last_error()
    for n in (1, 999, 50000):
        assert L.lq_la_workspace_bytes(ctypes.byref(c), 1, n, 100000) <= need


def test_single_token_arguments_refused(L):
    c = config(L)
    assert step(L, c, n=0) == lq.OK
    for kw in (dict(n=-1), dict(s=None), dict(s=S + 8), dict(q=None), dict(o=O + 2), dict(o=Q), dict(s=Q), dict(s=O),
               dict(s=V), dict(s=A), dict(n=2**31)):
        assert step(L, c, **kw) == lq.ERR_INVALID_ARG, kw


def select(L, dtype=lq.BF16, batch=2, beams=4, vocab=1000, n_best=8, x=Q, stride=1000, s=K, os=V, op=A, ot=O, ws=WS,
           nbytes=1 << 40):
    return L.lq_beam_select(dtype, batch, beams, vocab, n_best, x, stride, s, os, op, ot, ws, nbytes, None)


def test_selection_arguments_refused(L):
    assert select(L, batch=0) == lq.OK
    for kw in (dict(dtype=5), dict(batch=-1), dict(beams=0), dict(beams=33), dict(vocab=0), dict(vocab=2**30),
               dict(n_best=0), dict(n_best=65), dict(vocab=1, beams=4, n_best=5), dict(stride=999), dict(x=None),
               dict(x=Q + 1), dict(s=None), dict(s=K + 2), dict(os=None), dict(op=A + 1), dict(ot=None), dict(ws=None),
               dict(ws=WS + 64), dict(nbytes=100), dict(os=Q + 64), dict(op=V), dict(ot=A + 32), dict(ws=Q),
               dict(os=K), dict(batch=2**31)):
        assert select(L, **kw) == lq.ERR_INVALID_ARG, kw
        assert lq.last_error() != "", kw
    assert lq.beam_workspace_bytes(2, 40, 1000, 8) == 0
    assert lq.beam_workspace_bytes(2, 4, 1000, 8) > 0


def test_reordering_arguments_refused(L):
    cfg = lq.config()
    state = 1 << 34

    def call(n=24, outer=2, groups=3, beams=4, inner=1, st=state, p=Q, c=cfg):
        return L.lq_state_reorder(ctypes.byref(c), st, n, outer, groups, beams, inner, p, None)

    def call32(n=24, outer=2, groups=3, beams=4, inner=1, st=S, p=Q):
        return L.lq_fp32_state_reorder(st, n, outer, groups, beams, inner, p, None)

    for f in (call, call32):
        assert f(n=0, groups=0) == lq.OK
        for kw in (dict(n=23), dict(n=-1), dict(beams=0, n=0), dict(beams=33, n=198), dict(outer=-1), dict(inner=2),
                   dict(st=None), dict(p=None), dict(p=Q + 2), dict(outer=2**31 - 1, groups=2**31 - 1, inner=2**31 - 1),
                   dict(outer=2**40), dict(n=0)):
            assert f(**kw) == lq.ERR_INVALID_ARG, kw
    assert call(st=state + 128) == lq.ERR_INVALID_ARG
    assert call(p=state + 512) == lq.ERR_INVALID_ARG
    assert call32(st=S + 8) == lq.ERR_INVALID_ARG and call32(p=S + 65536) == lq.ERR_INVALID_ARG
    bad = lq.config(window=99)
    assert call(c=bad) == lq.ERR_UNSUPPORTED


def test_plain_forms_on_hand_worked_values():
    """The references themselves: two tokens of one head, a two-beam choice, a swap."""
    q = np.zeros((2, 1, 128)); k = q.copy(); v = q.copy()
    k[0, 0, 0] = k[1, 0, 1] = 1.0
    v[0, 0, 0] = v[1, 0, 0] = 2.0
    q[:, 0, :2] = 1.0
    o, S = la_reference(q, k, v, np.array([[0.5], [0.25]]), [2])
    assert o[0, 0, 0] == 2.0 and o[1, 0, 0] == 2.5 and S[0, 0, 0, 0] == 0.5 and S[0, 0, 0, 1] == 2.0
    s, p, t = beam_reference(np.log(np.array([[[0.5, 0.5], [0.9, 0.1]]])), np.array([[0.0, -0.1]]), 3)
    assert p.tolist() == [[1, 0, 0]] and t.tolist() == [[0, 0, 1]]
    planes = {"counts": np.array([1, 2]), "rec_k": np.arange(8.0).reshape(2, 2, 2), "x": np.array([[1.0], [2.0]])}
    out = reorder_reference(planes, np.array([[1, 0]]), 1, 1, counts=planes["counts"])
    assert out["counts"].tolist() == [2, 1] and out["x"].tolist() == [[2.0], [1.0]]
    assert out["rec_k"].tolist() == [[[4, 5], [6, 7]], [[0, 1], [6, 7]]]
