"""The target-pass entry points check their arguments on the host, before
touching the device, and the binding's structs match the header's."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOME = ctypes.c_void_p(16)


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_drafter_markov_gb300 import _lib
    return _lib


def test_struct_layouts_match_header(lib, tmp_path):
    structs = {"page_map": lib.PageMapArgs, "cache_store": lib.CacheStoreArgs, "tree_attention": lib.TreeAttentionArgs,
               "logit_rules": lib.LogitRulesArgs}
    fields = [(f"dspark_{n}_args", cls, f[0]) for n, cls in structs.items() for f in cls._fields_]
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "dspark.h"\nint main(void){'
                   + "".join(f'printf("%zu ", sizeof(dspark_{n}_args));' for n in structs)
                   + "".join(f'printf("%zu ", offsetof({c}, {f}));' for c, _, f in fields) + "return 0;}\n")
    exe = tmp_path / "sizes"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert got == [ctypes.sizeof(c) for c in structs.values()] + [getattr(c, f).offset for _, c, f in fields]


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
    rc = getattr(L, fn)(ctypes.byref(a), *more)
    assert rc == code, L.dspark_last_error()
    assert L.dspark_last_error()


def test_null_structs(lib):
    L = lib.load()
    assert L.dspark_page_map(None, None) == lib.ERR_INVAL
    assert L.dspark_cache_store(None, None) == lib.ERR_INVAL
    assert L.dspark_tree_attention(None, None, None) == lib.ERR_INVAL
    assert L.dspark_tree_attention_workspace_size(None) == 0
    assert L.dspark_logit_rules(None, None) == lib.ERR_INVAL


def test_page_map_refusals(lib):
    good = dict(R=4, page=16, n_pages=100, max_pages=10, N=20, n_parents=20, W=1, held_out=ctypes.c_void_p(32),
                n_free_out=ctypes.c_void_p(48))
    for over, code in [(dict(R=0), 1), (dict(page=0), 1), (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(N=-1), 1),
                       (dict(R=8193), 6), (dict(n_pages=1 << 30), 6), (dict(table=None), 1), (dict(slot=None), 1),
                       (dict(mask=None), 1), (dict(parents=None), 1), (dict(W=0), 1), (dict(n_parents=-1), 1),
                       (dict(held_out=SOME), 1), (dict(n_free_out=SOME), 1)]:
        refused(lib, "dspark_page_map", filled(lib.PageMapArgs, **{**good, **over}), code, None)


def test_cache_store_refusals(lib):
    good = dict(N=4, H=2, D=64, page=16, n_pages=10, dtype=1)
    for over, code in [(dict(N=-1), 1), (dict(H=0), 1), (dict(D=0), 1), (dict(page=0), 1), (dict(n_pages=0), 1), (dict(dtype=2), 1),
                       (dict(H=1 << 11, D=1 << 10), 6), (dict(k=None), 1), (dict(slot=None), 1)]:
        refused(lib, "dspark_cache_store", filled(lib.CacheStoreArgs, **{**good, **over}), code, None)
    a = filled(lib.CacheStoreArgs, **{**good, "N": 0, "k": None})
    assert lib.load().dspark_cache_store(ctypes.byref(a), None) == lib.OK  # nothing to write: no launch


def test_tree_attention_refusals(lib):
    good = dict(R=4, N=8, Hq=8, H=2, D=64, page=16, n_pages=10, max_pages=4, dtype=1, W=1, max_rows=4, scale=1.0)
    for over, code in [(dict(R=0), 1), (dict(N=-1), 1), (dict(H=0), 1), (dict(Hq=9), 1), (dict(Hq=1), 1), (dict(D=0), 1),
                       (dict(D=257), 6), (dict(page=0), 1), (dict(max_pages=0), 1), (dict(dtype=7), 1), (dict(W=0), 1),
                       (dict(max_rows=0), 1), (dict(n_pages=1 << 30), 6), (dict(max_pages=1 << 28), 6), (dict(q=None), 1),
                       (dict(table=None), 1), (dict(out=None), 1)]:
        refused(lib, "dspark_tree_attention", filled(lib.TreeAttentionArgs, **{**good, **over}), code, SOME, None)
    a = filled(lib.TreeAttentionArgs, **good)
    refused(lib, "dspark_tree_attention", a, 1, None, None)  # no workspace
    a.N = 0
    assert lib.load().dspark_tree_attention(ctypes.byref(a), None, None) == lib.OK


def test_logit_rules_refusals(lib):
    good = dict(R=4, N=8, V=100, dtype=1, max_hist=5, n_bias=3, n_allow=2, W=1)
    for over, code in [(dict(R=0), 1), (dict(N=-1), 1), (dict(V=0), 1), (dict(dtype=5), 1), (dict(R=65536), 6), (dict(T=None), 1),
                       (dict(row_start=None), 1), (dict(hist_len=None), 1), (dict(bias_id=None), 1), (dict(allow_row=None), 1),
                       (dict(W=0), 1), (dict(max_hist=-1), 1)]:
        refused(lib, "dspark_logit_rules", filled(lib.LogitRulesArgs, **{**good, **over}), code, None)


def test_tables_whose_last_tile_passes_32_bits_are_refused(lib):
    a = filled(lib.TreeAttentionArgs, R=4, N=8, Hq=8, H=2, D=64, page=16, n_pages=10, max_pages=(1 << 27) - 1, dtype=1, W=1,
               max_rows=4, scale=1.0)
    refused(lib, "dspark_tree_attention", a, lib.ERR_UNSUPPORTED, SOME, None)
