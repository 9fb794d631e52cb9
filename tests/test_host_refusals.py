"""A workspace that the kernels could not address, and a machine without a GPU, are
errors that the host returns."""
import ctypes

import pytest
import torch

SOME = ctypes.c_void_p(256)


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_drafter_markov_gb300 import _lib
    return _lib


def filled(cls, **over):
    a = cls()
    for name, kind in cls._fields_:
        if kind is ctypes.c_void_p:
            setattr(a, name, SOME)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def calls(lib):
    draft = filled(lib.DraftArgs, R=4, gamma=4, V=100, r=8, d=8, dtype=1)
    rnn = filled(lib.RnnArgs, base=draft)
    yield "dspark_draft_markov", draft, ()
    yield "dspark_draft_markov_step", draft, (1,)
    yield "dspark_draft_rnn", rnn, ()
    yield "dspark_verify", filled(lib.VerifyArgs, R=4, gamma=4, V=100, r=8, dtype=1, N=20), ()
    yield "dspark_sts_fit", filled(lib.StsArgs, M=16, gamma=4, G=8, n_bins=10), ()
    yield "dspark_tree_attention", filled(lib.TreeAttentionArgs, R=4, N=8, Hq=8, H=2, D=64, page=16, n_pages=10, max_pages=4, dtype=1,
                                          W=1, max_rows=4, scale=1.0), ()


@pytest.mark.skipif(torch.cuda.is_available(), reason="pointers that are not memory: for a machine without a GPU")
def test_refused_by_every_call(lib):
    L = lib.load()
    for name, a, more in calls(lib):
        for ws in (257, 260, 264, 0):
            assert getattr(L, name)(ctypes.byref(a), *more, ctypes.c_void_p(ws), None) == lib.ERR_INVAL, (name, ws)
            assert b"workspace" in L.dspark_last_error(), name


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_views_off_the_boundary_are_refused(lib, dtype):
    from test_gpu_target import call, check, make
    s = make([700, 30], [3, 2], 8, 2, 128, 16, dtype, seed=1)
    out, err = call(s)
    check(s, out, err)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")  # 40 MB are the most that a call needs
    for off in (1, 4, 8):
        with pytest.raises(lib.DSparkError, match="workspace"):
            call(s, ws=ws[off:])
    same, err = call(s, ws=ws[16:])
    assert torch.equal(same["out"], out["out"])


@pytest.mark.skipif(torch.cuda.is_available(), reason="pointers that are not memory: for a machine without a GPU")
def test_no_gpu_is_an_error_code(lib):
    """Arguments that pass every check, on a machine without a GPU."""
    L = lib.load()
    for name, a, more in calls(lib):
        assert getattr(L, name)(ctypes.byref(a), *more, SOME, None) == lib.ERR_CUDA, name
    for name, a in (("dspark_page_map", filled(lib.PageMapArgs, R=4, page=16, n_pages=100, max_pages=10, N=20, n_parents=20, W=1,
                                               held_out=ctypes.c_void_p(512), n_free_out=ctypes.c_void_p(768))),
                    ("dspark_cache_store", filled(lib.CacheStoreArgs, N=4, H=2, D=64, page=16, n_pages=10, dtype=1)),
                    ("dspark_logit_rules", filled(lib.LogitRulesArgs, R=4, N=8, V=100, dtype=1, max_hist=5, n_bias=3, n_allow=2, W=1))):
        assert getattr(L, name)(ctypes.byref(a), None) == lib.ERR_CUDA, name
    for dtype, D in ((0, 64), (1, 200), (0, 3)):  # the other two kernels of the attention
        a = filled(lib.TreeAttentionArgs, R=4, N=8, Hq=8, H=2, D=D, page=16, n_pages=10, max_pages=4, dtype=dtype, W=1, max_rows=4, scale=1.0)
        assert L.dspark_tree_attention(ctypes.byref(a), SOME, None) == lib.ERR_CUDA, (dtype, D)
