"""lq_la_prefill refuses every pair of buffers of which one is written and the other read or written (no GPU: addresses
stand in for buffers)."""
import ctypes

import pytest

from quantized_linear_attention_gb300 import build as lq_build
from quantized_linear_attention_gb300 import lq

GB = 1 << 30
PLACES = {name: (i + 1) * 64 * GB for i, name in enumerate(["q", "k", "v", "alpha", "o", "S0", "S_out", "workspace", "cu"])}
SEQS, TOKENS, LONGEST, HEADS = 3, 9000, 4000, 2  # split in every type


@pytest.fixture(scope="module")
def L():
    lq_build.build_lq()
    return lq.load()


def call(L, dtype, **at):
    c = lq.LaConfig()
    L.lq_la_config_default(ctypes.byref(c), HEADS, 1, dtype)
    a = dict(PLACES, **at)
    rc = L.lq_la_prefill(ctypes.byref(c), SEQS, TOKENS, LONGEST, a["cu"], a["q"], a["k"], a["v"], a["alpha"], a["S0"],
                         a["S_out"], a["o"], a["workspace"], 1 << 40, None)
    return rc, lq.last_error()


@pytest.mark.parametrize("dtype", [lq.BF16, lq.F16, lq.F32])
@pytest.mark.parametrize("written", ["o", "S_out", "workspace"])
def test_no_written_buffer_may_overlap_another(L, dtype, written):
    for other in PLACES:
        if other == written or {other, written} == {"S0", "S_out"}:
            continue
        for shift in (0, 256):  # the other one begins inside, or this one does
            for who, where in ((other, written), (written, other)):
                rc, error = call(L, dtype, **{who: PLACES[where] + shift})
                # cu_seqlens is 16 bytes long: nothing begins 256 bytes into it
                if where == "cu" and shift:
                    continue
                assert rc == lq.ERR_INVALID_ARG and "overlap" in error, (who, where, shift, rc, error)
    rc, error = call(L, dtype, S_out=PLACES["S0"] + 4096)
    assert rc == lq.ERR_INVALID_ARG and "overlap" in error


@pytest.mark.parametrize("dtype", [lq.BF16, lq.F16, lq.F32])
def test_what_may_be_shared(L, dtype):
    """S_out may be S0, and inputs may be one another: these get as far as the device's checks."""
    for at in (dict(), dict(S_out=PLACES["S0"]), dict(k=PLACES["q"]), dict(alpha=PLACES["S0"]), dict(v=PLACES["k"] + 256)):
        rc, error = call(L, dtype, **at)
        assert "overlap" not in error, (at, error)
