"""The attention's index arithmetic (csrc/attn_cut.h) at the ends of its ranges, on
the CPU: the header is compiled by g++ into small programs."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_drafter_markov_gb300", "csrc")


def run(tmp_path, source, *args):
    src, exe = tmp_path / "cut.cpp", tmp_path / "cut"
    src.write_text(source)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I", CSRC,
                           "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    return subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True)


LOOKUP = r"""
#include "attn_cut.h"
#include <cstdio>
#include <cstdlib>
using namespace dspark::attn;
// every lane of every tile near the end of a table of max_pages pages: the entry that
// it looks up is one of the request's, and of its box where the box has tokens
int main(int, char **v) {
    const int page = atoi(v[1]), max_pages = atoi(v[2]), tokens = atoi(v[3]), cols = atoi(v[4]), log2 = 7, tile = 1 << log2;
    const int last = tokens - 1, tiles = (int)(((unsigned)tokens + tile - 1) >> log2);
    int box = page & -page;
    if (box > tile) box = tile;
    for (int t = tiles > 40 ? tiles - 40 : 0; t < tiles; ++t)
        for (int lane = 0; lane < 32; ++lane) {
            const int b = lane / cols, tok = lookup_token(t, log2, b, box, last), entry = tok / page;
            if (tok < 0 || entry < 0 || entry >= max_pages || entry > last / page) return printf("tile %d lane %d: token %d", t, lane, tok), 1;
            const long long first = (long long)t * tile + (long long)b * box;
            if (b * box < tile && first <= last && tok != first) return printf("tile %d lane %d: token %d, not %lld", t, lane, tok, first), 1;
        }
    return 0;
}
"""


@pytest.mark.parametrize("cols", [1, 2])
@pytest.mark.parametrize("page,max_pages", [(45691136, 47), (256, 8388607), (16, 134217712), (128, 16777214), (8, 268435424), (48, 44739237)])
def test_table_lookups_stay_in_the_row(tmp_path, page, max_pages, cols):
    """Requests whose tokens end just below 2^31, the most that a table may name."""
    assert page * max_pages <= 0x7fffff00
    for short in (0, 1, 100, 129, 3000):
        r = run(tmp_path, LOOKUP, page, max_pages, page * max_pages - short, cols)
        assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("page,tokens", [(16, 1), (16, 128), (8, 777), (40, 1000), (1024, 5000)])
def test_table_lookups_of_small_requests(tmp_path, page, tokens):
    r = run(tmp_path, LOOKUP, page, (tokens + page - 1) // page, tokens, 2)
    assert r.returncode == 0, r.stdout + r.stderr
