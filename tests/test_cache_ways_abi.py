"""Entry points around the cache -- rope_store, cache_store4, tree_attention4 -- check
their arguments on the host, before touching the device, and the binding's structs match
the header's."""
import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOME = ctypes.c_void_p(256)


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_drafter_markov_gb300 import _lib
    return _lib


def test_struct_layouts_match_header(lib, tmp_path):
    structs = {"rope_store": lib.RopeStoreArgs, "cache_store4": lib.CacheStore4Args}
    fields = [(f"dspark_{n}_args", f[0]) for n, cls in structs.items() for f in cls._fields_]
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dspark.h"\nint main(void){'
                   + "".join(f'printf("%zu ", sizeof(dspark_{n}_args));' for n in structs)
                   + "".join(f'printf("%zu ", offsetof({c}, {f}));' for c, f in fields) + "return 0;}\n")
    exe = tmp_path / "sizes"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert got == [ctypes.sizeof(c) for c in structs.values()] + [getattr(c, f[0]).offset for c in structs.values() for f in c._fields_]


def filled(cls, **over):
    a = cls()
    for name, kind in cls._fields_:
        if kind is ctypes.c_void_p:
            setattr(a, name, SOME)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def refused(lib, fn, a, code, *more):
    L = lib.load()
    assert getattr(L, fn)(ctypes.byref(a), *more) == code, L.dspark_last_error()
    assert L.dspark_last_error()


ROPE = dict(N=4, Hq=8, H=2, D=64, rot=64, page=16, n_pages=10, dtype=1, eps=1e-6)
STORE = dict(N=4, H=2, D=64, page=16, n_pages=10, dtype=1)
ATTN = dict(R=4, N=8, Hq=8, H=2, D=64, page=16, n_pages=10, max_pages=4, dtype=1, W=1, max_rows=4, scale=1.0)


def test_null_structs(lib):
    L = lib.load()
    assert L.dspark_rope_store(None, None) == lib.ERR_INVAL
    assert L.dspark_cache_store4(None, None) == lib.ERR_INVAL
    assert L.dspark_tree_attention4(None, None, None) == lib.ERR_INVAL
    assert L.dspark_tree_attention4_workspace_size(None) == 0


def test_rope_store_refusals(lib):
    for over, code in [(dict(N=-1), 1), (dict(Hq=-1), 1), (dict(H=-1), 1), (dict(Hq=0, H=0), 1), (dict(q=None, k=None), 1), (dict(D=0), 1),
                       (dict(D=257, rot=0), 6), (dict(dtype=2), 1), (dict(rot=-2), 1), (dict(rot=63), 1), (dict(rot=66), 1), (dict(eps=0.0), 1),
                       (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(Hq=1 << 15), 6), (dict(page=0), 1),
                       (dict(n_pages=0), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(pos=None), 1), (dict(freq=None), 1), (dict(q_out=None), 1),
                       (dict(k_cache=None), 1), (dict(v_cache=None), 1), (dict(slot=None, k_out=None), 1)]:
        refused(lib, "dspark_rope_store", filled(lib.RopeStoreArgs, **{**ROPE, **over}), code, None)
    a = filled(lib.RopeStoreArgs, **{**ROPE, "N": 0, "pos": None})
    assert lib.load().dspark_rope_store(ctypes.byref(a), None) == lib.OK  # no rows: no launch


def test_cache_store4_refusals(lib):
    for over, code in [(dict(N=-1), 1), (dict(H=0), 1), (dict(D=0), 1), (dict(page=0), 1), (dict(n_pages=0), 1), (dict(dtype=2), 1),
                       (dict(D=72), 6), (dict(D=272), 6), (dict(page=1), 6), (dict(D=16, page=4), 6), (dict(H=1 << 15), 6), (dict(k=None), 1),
                       (dict(v=None), 1), (dict(slot=None), 1), (dict(k_cache=None), 1), (dict(k_out=None), 1), (dict(v_out=None), 1),
                       (dict(k_cache=ctypes.c_void_p(264)), 1), (dict(v_cache=ctypes.c_void_p(8)), 1), (dict(k_out=ctypes.c_void_p(258)), 1)]:
        refused(lib, "dspark_cache_store4", filled(lib.CacheStore4Args, **{**STORE, **over}), code, None)
    a = filled(lib.CacheStore4Args, **{**STORE, "N": 0, "k": None})
    assert lib.load().dspark_cache_store4(ctypes.byref(a), None) == lib.OK


def test_tree_attention4_refusals(lib):
    for over, code in [(dict(R=0), 1), (dict(N=-1), 1), (dict(H=0), 1), (dict(Hq=9), 1), (dict(Hq=1), 1), (dict(D=0), 1), (dict(D=272), 6),
                       (dict(D=40), 6), (dict(page=0), 1), (dict(page=1), 6), (dict(max_pages=0), 1), (dict(dtype=7), 1), (dict(W=0), 1),
                       (dict(W=5), 6), (dict(max_rows=0), 1), (dict(n_pages=1 << 30), 6), (dict(max_pages=1 << 28), 6), (dict(q=None), 1),
                       (dict(k_cache=None), 1), (dict(v_cache=ctypes.c_void_p(260)), 1), (dict(table=None), 1), (dict(out=None), 1)]:
        a = filled(lib.TreeAttentionArgs, **{**ATTN, **over})
        refused(lib, "dspark_tree_attention4", a, code, SOME, None)
    a = filled(lib.TreeAttentionArgs, **ATTN)
    refused(lib, "dspark_tree_attention4", a, 1, None, None)  # no workspace
    refused(lib, "dspark_tree_attention4", a, 1, ctypes.c_void_p(264), None)
    a.N = 0
    assert lib.load().dspark_tree_attention4(ctypes.byref(a), None, None) == lib.OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="pointers that are not memory: for a machine without a GPU")
def test_no_gpu_is_an_error_code(lib):
    L = lib.load()
    for D in (64, 9):
        a = filled(lib.RopeStoreArgs, **{**ROPE, "D": D, "rot": 8})
        assert L.dspark_rope_store(ctypes.byref(a), None) == lib.ERR_CUDA
    assert L.dspark_cache_store4(ctypes.byref(filled(lib.CacheStore4Args, **STORE)), None) == lib.ERR_CUDA
    for dtype, D in ((1, 64), (0, 64), (1, 256)):
        a = filled(lib.TreeAttentionArgs, **{**ATTN, "dtype": dtype, "D": D})
        assert L.dspark_tree_attention4(ctypes.byref(a), SOME, None) == lib.ERR_CUDA
