"""Rows of which a grammar allows nothing, from the rules into the verification:
reported, token 0, and nothing else is touched."""
import numpy as np
import pytest
import torch

from parity import host
from speculative_decoding_drafter_markov_gb300 import _lib as dsp
from speculative_decoding_drafter_markov_gb300 import workloads as W
from test_gpu_verify import _case

pytestmark = pytest.mark.gpu


def _verify(inp, x, logq, lse, tags, T, seed, cycle):
    dev = lambda a: torch.as_tensor(a, device="cuda")  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = dsp.verify(T, dev(tags), inp["anchor"].cuda(), dev(x), dev(logq), dev(lse), inp["U"].cuda(), inp["W1"].cuda(),
                     inp["W2t"].cuda(), seed=seed, cycle=cycle, err=err)
    return {k: host(v) for k, v in out.items()}, int(err)


@pytest.mark.parametrize("wl", [W.small("qwen4b", R=24, gamma=5, V=5000, r=64, d=32),              # tensor cores
                                W.small("qwen4b", R=9, gamma=4, V=1001, r=24, d=40, dtype="f32")],  # CUDA cores
                         ids=lambda w: w.dtype)
def test_rows_that_allow_nothing(orc, wl):
    rng = np.random.default_rng(5)
    ell = rng.integers(0, wl.gamma + 1, wl.R)
    ell[:3] = 0, wl.gamma, 2
    inp, x, logq, lse, _, tags, T = _case(orc, wl, 31, 4, ell)
    T = T.cuda()
    start = np.concatenate([[0], np.cumsum(ell + 1)]).astype(np.int32)
    good, err = _verify(inp, x, logq, lse, tags, T, 31, 4)
    assert err == 0
    # the only row of request 0, the first of request 1, and the last of one that accepts everything
    whole = [r for r in range(2, wl.R) if good["n_accept"][r] == ell[r]]
    closed = {0: 0, 1: 0, whole[0]: int(ell[whole[0]])}
    allow_row = torch.full((T.shape[0],), -1, dtype=torch.int32, device="cuda")
    for r, j in closed.items():
        allow_row[start[r] + j] = 0
    none = torch.zeros((1, (wl.V + 31) // 32), dtype=torch.int32, device="cuda")
    rules_err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ruled = dsp.logit_rules(T, torch.from_numpy(start).cuda(), allow=none, allow_row=allow_row, err=rules_err)
    rows = [int(start[r] + j) for r, j in closed.items()]
    assert int(rules_err) == 0 and bool(torch.isneginf(ruled[rows].float()).all())
    got, err = _verify(inp, x, logq, lse, tags, ruled, 31, 4)
    assert err == dsp.ERR_NONFINITE
    assert np.isneginf(got["lse_p"][rows]).all()
    for r in range(wl.R):
        if r not in closed:
            for k in ("n_accept", "out_tokens", "next_anchor"):
                assert np.array_equal(got[k][r], good[k][r]), (k, r)
            keep = slice(start[r], start[r + 1])
            assert np.array_equal(got["lse_p"][keep], good["lse_p"][keep])
        else:
            n = closed[r]
            assert got["n_accept"][r] == n and got["next_anchor"][r] == 0
            assert got["out_tokens"][r].tolist() == x[r, :n].tolist() + [0] + [-1] * (wl.gamma - n)
