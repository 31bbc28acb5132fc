"""Workspaces of split scans for every class of state counts (host only): the query for the largest call is enough for
every smaller one."""
import ctypes
import random

import pytest

from quantized_linear_attention_gb300 import build as lq_build
from quantized_linear_attention_gb300 import lq
from tests.test_layers_cpu import ssm, ssm_cfg


@pytest.fixture(scope="module")
def L():
    lq_build.build_lq()
    return lq.load()


@pytest.mark.parametrize("n_state", [5, 8, 12, 16, 17, 20, 32, 33, 48])
def test_the_largest_call_s_workspace_is_enough(L, n_state):
    rng, split = random.Random(n_state), 0
    for channels in (16, 64, 513, 4096):
        c = ssm_cfg(L, channels, n_state, 1)
        for n_seqs, n, m in ((1, 100000, 0), (16, 20000, 3000), (3, 700, 300), (200, 5000, 0)):
            most = L.lq_ssm_workspace_bytes(ctypes.byref(c), n_seqs, n, m)
            for i in range(200):
                s, t = (n_seqs, n) if i == 0 else (rng.randint(1, n_seqs), rng.randint(0, n))
                k = rng.choice([m, rng.randint(1, m or n)])
                ssm(L, c, n_seqs=s, n_tokens=t, max_len=k, nbytes=0)
                e = lq.last_error()
                if "are needed" in e:
                    split += 1
                    assert int(e.split(", ")[1].split()[0]) <= most, (channels, n_state, s, t, k)
    assert split > 100
