"""lq_la_workspace_bytes for the largest call is enough for every smaller one (no GPU: addresses stand in for buffers,
and a call with too little workspace says how much it needs)."""
import ctypes
import random
import re

import pytest

from quantized_linear_attention_gb300 import build as lq_build
from quantized_linear_attention_gb300 import lq

GB = 1 << 30
Q, K, V, A, O, S0, S, WS, CU = ((i + 1) * 1024 * GB for i in range(9))


@pytest.fixture(scope="module")
def L():
    lq_build.build_lq()
    return lq.load()


def config(L, dtype, heads):
    c = lq.LaConfig()
    L.lq_la_config_default(ctypes.byref(c), heads, 1, dtype)
    return c


def needed(L, c, n_seqs, n_tokens, max_len):
    """What the call itself asks for; 0 where it gets past its workspace."""
    L.lq_la_prefill(ctypes.byref(c), n_seqs, n_tokens, max_len, CU, Q, K, V, A, S0, S, O, WS, 0, None)
    m = re.search(r"workspace has 0 bytes, (\d+) are needed", lq.last_error())
    return int(m.group(1)) if m else 0


def query(L, c, n_seqs, n_tokens, max_len):
    return L.lq_la_workspace_bytes(ctypes.byref(c), n_seqs, n_tokens, max_len)


DTYPES = [lq.BF16, lq.F16, lq.F32]


@pytest.mark.parametrize("dtype,heads,n_seqs,max_len,large,small", [
    (lq.BF16, 32, 16, 2000, 100000, 5000), (lq.F32, 1, 1, 100000, 100000, 39168)])
def test_a_smaller_call_that_is_split_more(L, dtype, heads, n_seqs, max_len, large, small):
    c = config(L, dtype, heads)
    assert needed(L, c, n_seqs, small, max_len) > needed(L, c, n_seqs, large, max_len)
    assert query(L, c, n_seqs, large, max_len) >= needed(L, c, n_seqs, small, max_len)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", [1, 2, 3, 7, 17, 32, 94, 95, 96, 100, 151, 152, 153, 189, 190, 191, 192, 400])
def test_smaller_calls_never_need_more(L, dtype, heads):
    """Fewer tokens, fewer sequences, a shorter longest one: every length near where the plan changes, and random ones."""
    c, rng = config(L, dtype, heads), random.Random(heads)
    for n_seqs, large, max_len in [(1, 400000, 0), (1, 3000, 0), (16, 100000, 2000), (3, 700, 300), (64, 20000, 1025),
                                   (5, 2000000, 30000)]:
        most = query(L, c, n_seqs, large, max_len)
        sizes = set(range(250, min(large, 420))) | {x + d for x in (1024, 2048, 1500, max_len) for d in range(-2, 4)}
        for seg in list(range(128, 1025, 16)) + list(range(512, 8192, 128)):  # where a segment grows by a step
            for pieces in (304, 304 - heads, 152):
                sizes |= {max(1, seg * pieces // heads + d) for d in (-1, 0, 1, pieces // heads)}
        sizes |= {rng.randint(1, large) for _ in range(300)}
        for n in sorted(s for s in sizes if 0 <= s <= large):
            assert needed(L, c, n_seqs, n, max_len) <= most, (n_seqs, n, max_len)
        assert needed(L, c, n_seqs, large, max_len) <= most
        for _ in range(200):
            m = rng.randint(1, max_len or large)
            assert needed(L, c, rng.randint(1, n_seqs), rng.randint(1, large), m) <= most


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_more_than_the_largest_call_could_need(L, dtype):
    """None where no call up to this size is split, and never more than some call up to it needs, to two segments a head."""
    slack = 2 * 65536 + 3 * 256
    for heads, n_seqs, n, max_len in [(32, 1, 1000, 0), (4, 8, 100000, 256), (96, 4, 100000, 2048)]:
        if dtype == lq.BF16 or max_len == 256:
            assert query(L, config(L, dtype, heads), n_seqs, n, max_len) == 0
    for heads, n_seqs, n in [(1, 1, 200000), (32, 16, 100000), (16, 4, 9000)]:
        c = config(L, dtype, heads)
        most = max(needed(L, c, n_seqs, x, 0) for x in range(256, n + 1, max(1, n // 4000)))
        assert query(L, c, n_seqs, n, 0) <= most + slack * heads
