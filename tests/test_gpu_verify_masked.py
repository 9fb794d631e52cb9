"""GPU parity of verification with target logits at -inf (tokens that a grammar
forbids): only allowed tokens come out, the others have probability zero."""
import numpy as np
import pytest
import torch

from parity import compare_verify, host
from speculative_decoding_drafter_markov_gb300 import workloads as W
from test_gpu_verify import _case, _gpu_verify, _oracle_verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wl", [W.small("qwen4b", R=24, gamma=5, V=5000, r=64, d=32),              # tensor cores
                                W.small("qwen4b", R=9, gamma=4, V=1001, r=24, d=40, dtype="f32")],  # CUDA cores
                         ids=lambda w: w.dtype)
@pytest.mark.parametrize("keep", [0.002, 0.3])
def test_forbidden_tokens(orc, wl, keep):
    rng = np.random.default_rng(int(keep * 1000))
    ell = rng.integers(0, wl.gamma + 1, wl.R)
    inp, x, logq, lse, A, tags, T = _case(orc, wl, 21, 2, ell)
    allow = rng.random(T.shape) < keep
    for i, (rq, j) in enumerate(tags):
        allow[i, rng.integers(0, wl.V)] = True
        if rng.random() < 0.5 and j < wl.gamma:  # often the drafted token is allowed
            allow[i, x[rq, j]] = True
    T = torch.where(torch.from_numpy(allow), T.float(), torch.tensor(-float("inf"))).to(T.dtype)
    got = _gpu_verify(inp, x, logq, lse, A, tags, T, 21, 2)
    ref = _oracle_verify(orc, inp, x, logq, lse, A, tags, T, 21, 2)
    # a forbidden drafted token has log p = -inf on both sides; the rest as ever
    never = np.isneginf(ref["logp"])
    assert np.array_equal(np.isneginf(got["logp"]), never) and never.any()
    got["logp"], ref["logp"] = (np.where(never, 0.0, v["logp"]) for v in (got, ref))
    compare_verify(got, ref, list(range(wl.R)), tags, wl.gamma)
    row = 0
    for rq in range(wl.R):
        n = int(got["n_accept"][rq])
        for j in range(n + 1):
            assert allow[row + j, got["out_tokens"][rq, j]]
        row += int(ell[rq]) + 1
