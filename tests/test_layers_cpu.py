"""What the state space layer's calls and token_logprobs refuse, on the host (no GPU): addresses stand in for buffers."""
import ctypes
import random

import numpy as np
import pytest

from quantized_linear_attention_gb300 import build as lq_build
from quantized_linear_attention_gb300 import lq
from tests._layers import conv_reference, logprob_reference, ssm_reference

TB = 1 << 40
PLACES = {n: (i + 1) * TB for i, n in enumerate(
    ["x", "dt", "z", "B", "C", "y", "A", "D", "dt_bias", "S0", "S", "cu", "workspace", "weight", "bias", "logits", "tokens",
     "logprob", "entropy", "top_logprob", "top_token"])}
BAD = lq.ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    lq_build.build_lq()
    return lq.load()


def conv_cfg(L, channels=256, width=4, dtype=lq.BF16, silu=1, **kw):
    c = lq.ConvConfig()
    L.lq_conv_config_default(ctypes.byref(c), channels, width, dtype, silu)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def conv(L, c, n_seqs=3, n_tokens=100, max_len=0, **at):
    a = dict(PLACES, **at)
    return L.lq_conv_prefill(ctypes.byref(c) if c else None, n_seqs, n_tokens, max_len, a["cu"], a["x"], a["weight"],
                             a["bias"], a["S0"], a["S"], a["y"], None)


def conv_step(L, c, n=3, **at):
    a = dict(PLACES, **at)
    return L.lq_conv_decode_step(ctypes.byref(c) if c else None, a["S"], n, a["x"], a["weight"], a["bias"], a["y"], None)


def ssm_cfg(L, channels=256, n_state=16, groups=2, dtype=lq.BF16, softplus=1, **kw):
    c = lq.SsmConfig()
    L.lq_ssm_config_default(ctypes.byref(c), channels, n_state, groups, dtype, softplus)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def ssm(L, c, n_seqs=3, n_tokens=100, max_len=0, nbytes=TB, **at):
    a = dict(PLACES, **at)
    return L.lq_ssm_prefill(ctypes.byref(c) if c else None, n_seqs, n_tokens, max_len, a["cu"], a["x"], a["dt"], a["A"],
                            a["B"], a["C"], a["D"], a["z"], a["dt_bias"], a["S0"], a["S"], a["y"], a["workspace"], nbytes, None)


def ssm_step(L, c, n=3, **at):
    a = dict(PLACES, **at)
    return L.lq_ssm_decode_step(ctypes.byref(c) if c else None, a["S"], n, a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"],
                                a["z"], a["dt_bias"], a["y"], None)


def logprobs(L, dtype=lq.BF16, rows=3, vocab=1000, n_top=4, stride=1000, **at):
    a = dict(PLACES, **at)
    return L.lq_token_logprobs(dtype, rows, vocab, n_top, a["logits"], stride, a["tokens"], a["logprob"], a["entropy"],
                               a["top_logprob"], a["top_token"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(channels=0), BAD), (dict(channels=2**20 + 1), BAD), (dict(width=1), lq.ERR_UNSUPPORTED),
    (dict(width=5), lq.ERR_UNSUPPORTED), (dict(dtype=3), BAD), (dict(dtype=-1), BAD), (dict(silu=2), BAD),
    (dict(x_stride=255), BAD), (dict(y_stride=0), BAD), (dict(x_stride=2**41), BAD), (dict(y_stride=-256), BAD)])
def test_convolutions_refused(L, kw, code):
    c = conv_cfg(L, **kw)
    assert conv(L, c) == code and lq.last_error() != ""
    assert conv_step(L, c) == code


@pytest.mark.parametrize("kw,code", [
    (dict(channels=0, groups=1), BAD), (dict(n_state=0), lq.ERR_UNSUPPORTED), (dict(n_state=65), lq.ERR_UNSUPPORTED),
    (dict(groups=3), BAD), (dict(groups=0), BAD), (dict(dtype=9), BAD), (dict(softplus=-1), BAD), (dict(reserved=1), BAD),
    (dict(x_stride=255), BAD), (dict(dt_stride=0), BAD), (dict(z_stride=1), BAD), (dict(y_stride=128), BAD),
    (dict(b_stride=31), BAD), (dict(c_stride=16), BAD), (dict(b_stride=2**41), BAD)])
def test_scans_refused(L, kw, code):
    c = ssm_cfg(L, **kw)
    assert ssm(L, c) == code and lq.last_error() != ""
    assert ssm_step(L, c) == code
    assert L.lq_ssm_workspace_bytes(ctypes.byref(c), 1, 100000, 0) == 0


def test_sizes_and_addresses_refused(L):
    cc, sc = conv_cfg(L), ssm_cfg(L)
    assert conv(L, None) == BAD and conv_step(L, None) == BAD and ssm(L, None) == BAD and ssm_step(L, None) == BAD
    assert conv(L, cc, n_seqs=0) == lq.OK and ssm(L, sc, n_seqs=0) == lq.OK
    assert conv_step(L, cc, n=0) == lq.OK and ssm_step(L, sc, n=0) == lq.OK
    sizes = [dict(n_seqs=-1), dict(n_tokens=-1), dict(max_len=-1), dict(n_tokens=2**31), dict(n_seqs=2**31), dict(cu=None),
             dict(cu=None, n_seqs=1, max_len=50), dict(cu=PLACES["cu"] + 2)]
    for kw in sizes + [dict(x=None), dict(y=None), dict(weight=None), dict(x=PLACES["x"] + 1), dict(y=PLACES["y"] + 1),
                       dict(weight=PLACES["weight"] + 2), dict(bias=PLACES["bias"] + 2), dict(S0=PLACES["S0"] + 1),
                       dict(S=PLACES["S"] + 1)]:
        assert conv(L, cc, **kw) == BAD and lq.last_error() != "", kw
    for kw in sizes + [{n: None} for n in ("x", "dt", "B", "C", "y", "A")] + [{n: PLACES[n] + 1} for n in (
            "x", "dt", "z", "B", "C", "y", "A", "D", "dt_bias", "S0", "S")] + [{n: PLACES[n] + 2} for n in ("A", "D", "S0", "S")]:
        assert ssm(L, sc, **kw) == BAD and lq.last_error() != "", kw
    for kw in (dict(n=-1), dict(n=2**31), dict(S=None), dict(x=None), dict(y=None), dict(S=PLACES["S"] + 1)):
        assert conv_step(L, cc, **kw) == BAD, kw
        assert ssm_step(L, sc, **kw) == BAD, kw


def test_logprob_arguments_refused(L):
    assert logprobs(L, rows=0) == lq.OK
    for kw in (dict(dtype=5), dict(rows=-1), dict(rows=2**31), dict(vocab=0), dict(vocab=2**31), dict(n_top=-1),
               dict(n_top=33), dict(vocab=3, stride=3), dict(stride=999), dict(stride=2**41), dict(logits=None),
               dict(logits=PLACES["logits"] + 1), dict(tokens=None), dict(logprob=None), dict(top_logprob=None),
               dict(top_token=None), dict(n_top=0), dict(tokens=PLACES["tokens"] + 2), dict(entropy=PLACES["entropy"] + 2),
               dict(tokens=None, logprob=None, entropy=None, n_top=0, top_logprob=None, top_token=None)):
        assert logprobs(L, **kw) == BAD and lq.last_error() != "", kw


def overlapping(call, names, written, may=()):
    for w in written:
        for other in names:
            if other == w:
                continue
            for who, where in ((other, w), (w, other)):
                assert call(**{who: PLACES[where]}) == BAD or {w, other} == set(may), (who, where)
                if {w, other} != set(may):
                    assert "overlap" in lq.last_error(), (who, where, lq.last_error())
    if may:
        assert call(**{may[0]: PLACES[may[1]] + 16}) == BAD and "overlap" in lq.last_error()
        call(**{may[0]: PLACES[may[1]]})
        assert "overlap" not in lq.last_error()


def test_no_written_buffer_may_overlap_another(L):
    overlapping(lambda **kw: conv(L, conv_cfg(L), **kw), ["x", "y", "weight", "bias", "S0", "S", "cu"], ["y", "S"], ("S", "S0"))
    overlapping(lambda **kw: conv_step(L, conv_cfg(L), **kw), ["x", "y", "weight", "bias", "S"], ["y", "S"])
    names = ["x", "dt", "z", "B", "C", "y", "A", "D", "dt_bias", "S0", "S", "cu"]
    overlapping(lambda **kw: ssm(L, ssm_cfg(L), **kw), names, ["y", "S"], ("S", "S0"))
    overlapping(lambda **kw: ssm_step(L, ssm_cfg(L), **kw), [n for n in names if n not in ("S0", "cu")], ["y", "S"])
    overlapping(lambda **kw: logprobs(L, **kw), ["logits", "tokens", "logprob", "entropy", "top_logprob", "top_token"],
                ["logprob", "entropy", "top_logprob", "top_token"])


def test_inputs_may_be_one_another(L):
    for kw in (dict(dt=PLACES["x"]), dict(C=PLACES["B"]), dict(z=PLACES["x"] + 64), dict(D=PLACES["dt_bias"])):
        ssm(L, ssm_cfg(L), **kw)
        assert "overlap" not in lq.last_error(), kw


def test_split_scans_need_their_workspace(L):
    """Where a call is split it refuses a workspace that is too small, missing, unaligned or in the way, and the query for
    the largest call is enough for every smaller one."""
    rng = random.Random(1)
    for channels, n_state in ((64, 16), (4096, 16), (100, 64), (33, 1), (20000, 8)):
        c = ssm_cfg(L, channels, n_state, 1)
        for n_seqs, n, m in ((1, 100000, 0), (16, 20000, 3000), (3, 700, 300), (200, 5000, 0)):
            most = L.lq_ssm_workspace_bytes(ctypes.byref(c), n_seqs, n, m)
            for _ in range(200):
                s, t = rng.randint(1, n_seqs), rng.randint(0, n)
                k = rng.choice([m, rng.randint(1, m or n), 0 if m == 0 else m])
                ssm(L, c, n_seqs=s, n_tokens=t, max_len=k, nbytes=0)
                e = lq.last_error()
                if "are needed" in e:
                    assert int(e.split(", ")[1].split()[0]) <= most, (channels, n_state, s, t, k)
    c = ssm_cfg(L, 64, 16, 1)
    need = L.lq_ssm_workspace_bytes(ctypes.byref(c), 1, 100000, 0)
    ssm(L, c, n_seqs=1, n_tokens=100000, nbytes=0)
    if "are needed" not in lq.last_error():
        pytest.skip("no sequence is split")
    for kw in (dict(workspace=None), dict(workspace=PLACES["workspace"] + 16), dict(workspace=PLACES["y"]),
               dict(workspace=PLACES["S"]), dict(workspace=PLACES["x"]), dict(workspace=PLACES["cu"])):
        assert ssm(L, c, n_seqs=1, n_tokens=100000, nbytes=need, **kw) == BAD and "workspace" in lq.last_error(), kw


def test_plain_forms_on_hand_worked_values():
    y, S, _ = conv_reference(np.array([[1.0], [2.0]]), np.array([[10.0, 1.0]]), np.array([0.5]), [2], np.array([[[3.0]]]), False)
    assert y[:, 0].tolist() == [31.5, 12.5] and S.tolist() == [[[2.0]]]
    ln2 = np.log(2.0)
    y, S, _, _ = ssm_reference(np.array([[1.0], [1.0]]), np.array([[ln2], [ln2]]), np.array([[-1.0]]), np.ones((2, 1, 1)),
                               np.full((2, 1, 1), 2.0), [2], D=np.array([1.0]), S0=np.array([[[4.0]]]), plus=False)
    assert np.allclose(S, 1 + 1.5 * ln2) and np.allclose(y[:, 0], [2 * (2 + ln2) + 1, 2 * (1 + 1.5 * ln2) + 1])
    lp, H, tl, ti = logprob_reference(np.log(np.array([[0.5, 0.25, 0.25]])), np.array([1]), 2)
    assert np.allclose(lp, np.log(0.25)) and np.allclose(H, 1.5 * ln2) and ti.tolist() == [[0, 1]]
