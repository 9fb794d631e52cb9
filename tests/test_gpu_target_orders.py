"""Queries, keys and values whose heads or rows stand in another order in memory than
in the batch.  Tolerances as in test_gpu_target.py: the values are the same, so where
the same kernel takes them the bits are."""
import pytest
import torch

import speculative_decoding_drafter_markov_gb300 as dsp
from test_gpu_target import call, check, err_word, expect, ints, make

pytestmark = pytest.mark.gpu


def heads_first(x):
    """The same [N, H, D] view of memory laid out as [H, N, D]."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [[1], [3, 2, 40], [150, 9]])
def test_queries_by_heads(dtype, rows):
    s = make([300, 0, 77][:len(rows)], rows, 8, 2, 64, 16, dtype, seed=4)
    want = expect(s)
    plain, err = call(s)
    check(s, plain, err, want)
    s["q"] = heads_first(s["q"])
    assert sum(rows) == 1 or s["q"].stride(1) > s["q"].stride(0)
    got, err = call(s)
    check(s, got, err, want)
    assert torch.equal(got["out"], plain["out"]) and torch.equal(got["lse"], plain["lse"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_queries_of_one_head_for_all(dtype):
    """A stride of zero between the heads, and rows from the last to the first."""
    s = make([30, 150], [2, 3], 4, 2, 64, 16, dtype, seed=5)
    s["q"] = s["q"][:, :1].expand(-1, 4, -1)
    check(s, *call(s))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [1, 7, 500])
def test_keys_and_values_by_heads(dtype, N):
    H, D, page = 4, 64, 16
    g = torch.Generator(device="cuda").manual_seed(N)
    k, v = (torch.randn((N, H, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    slot = torch.randperm((N // page + 2) * page, generator=g, device="cuda")[:N].int()
    out = []
    for change in (lambda x: x, heads_first):
        kc, vc = (torch.zeros((N // page + 2, H, page, D), dtype=dtype, device="cuda") for _ in range(2))
        err = err_word()
        dsp.cache_store(change(k), change(v), slot, kc, vc, err=err)
        assert int(err) == 0
        out.append((kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*out))
    assert torch.equal(out[0][0][slot.long() // page, :, slot.long() % page], k)


def test_empty_batches():
    """Calls of no rows, with outputs of no rows."""
    kc = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    table, zero = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), ints([0, 0])
    start = ints([0, 0, 0])
    out = dsp.tree_attention(q, kc, kc, table, zero, start)
    assert out["out"].shape == (0, 4, 64) and out["lse"].shape == (0, 4)
    dsp.cache_store(q[:, :2], q[:, :2], ints([]), kc, kc)
    assert dsp.logit_rules(torch.zeros((0, 50), device="cuda"), start).shape == (0, 50)
    m = dsp.page_map(zero, zero, table, zero, ints([0, 1, 2, 3]), ints([4]), page=16, N=0)
    assert m["slot"].shape == (0,) and m["row_start"].tolist() == [0, 0, 0]
