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


# The cut: every CTA's pieces, walked as the kernels walk them.
CUT = r"""
#include "attn_cut.h"
#include <cstdio>
#include <cstdlib>
#include <map>
#include <vector>
using namespace dspark::attn;
struct Case : Cut {
    std::vector<Request> q;
    Request request(int r) const { return q[r]; }
};
#define CHECK(x, ...) if (!(x)) return printf("%s: ", #x), printf(__VA_ARGS__), 1
// kind H G masked grid R (len rows)*
int main(int, char **v) {
    Case p{};
    const int kind = atoi(v[1]), grid = atoi(v[5]), R = atoi(v[6]);
    p.H = atoi(v[2]), p.G = atoi(v[3]), p.masked = atoi(v[4]);
    if (kind < 2) {  // 16 lines: the general kernel's tiles of 32, the fp32 kernel's of 64
        p.heads = p.G < 16 ? p.G : 16;
        p.block_rows = 16 / p.heads;
        p.tile_log2 = 5 + kind, p.unit_cost = 1 + kind;
        p.small_rows = p.block_rows, p.small_places = p.large_places = div_by(1);
    } else {  // one operand of 128 lines or two, tiles of 128
        p.heads = p.G;
        p.small_rows = 128 / p.G, p.block_rows = p.small_rows * (kind - 1);
        p.tile_log2 = 7, p.unit_cost = 3;
        p.small_places = div_by(3), p.large_places = div_by(kind == 3 ? 5 : 3);
    }
    p.subs = (p.G + p.heads - 1) / p.heads, p.lines = p.block_rows * p.heads, p.ctas = div_by(grid);
    for (int r = 0, row = 0; r < R; ++r) {
        const int len = atoi(v[7 + 2 * r]), rows = atoi(v[8 + 2 * r]);
        p.q.push_back(Request{row, rows, len});
        row += rows;
    }
    long long total = 0;
    std::vector<long long> begin(R);
    for (int r = 0; r < R; ++r) begin[r] = total, total = add_places(total, request_places(p, p.q[r]));
    CHECK(total <= (long long)grid * kMostShare, "%lld", total);
    // the unit that the next piece has to be of, and how many of its tiles are done
    int r = 0, b = 0, h = 0, done = 0;
    auto skip = [&] { while (r < R && p.q[r].rows == 0) ++r; };
    skip();
    long long expected = 0, most = 0, least_places = total;
    int open = 0;  // pieces of the unit so far
    Join join{};
    for (int c = 0; c < grid; ++c) {
        Share s = share_places(p, total, c, grid);
        if (s.n == 0) continue;
        CHECK(s.lo == expected && s.n > 0 && s.n <= kMostShare, "CTA %d begins at %lld, not %lld", c, s.lo, expected);
        expected += s.n;
        most = s.n > most ? s.n : most, least_places = s.n < least_places ? s.n : least_places;
        while (s.r + 1 < R && s.lo >= begin[s.r + 1]) ++s.r;
        s.r_begin = begin[s.r];
        Walk<Case> walk(p, s);
        Piece x;
        int pieces = 0;
        while (walk.next(x)) {
            const Request &q = p.q[r];
            CHECK(r < R && x.r == r && x.first == b * p.block_rows && x.head == h, "CTA %d: unit (%d, %d, %d), not (%d, %d, %d)", c, x.r,
                  x.first, x.head, r, b * p.block_rows, h);
            const int n = q.rows - x.first < p.block_rows ? q.rows - x.first : p.block_rows;
            const long long tokens = q.len + (long long)(p.masked ? q.rows : x.first + n);
            CHECK(x.n == n && x.tokens == tokens && x.row0 == q.row0 && x.rows == q.rows && x.len == q.len, "CTA %d", c);
            CHECK(x.tiles == (tokens + (1 << p.tile_log2) - 1) >> p.tile_log2, "CTA %d", c);
            CHECK(x.t0 == done && x.t0 < x.t1 && x.t1 <= x.tiles, "CTA %d: tiles %d .. %d after %d of %d", c, x.t0, x.t1, done, x.tiles);
            CHECK((x.slot < 0) == (x.t0 == 0 && x.t1 == x.tiles), "CTA %d", c);
            if (x.slot >= 0) {
                CHECK(x.slot == 2 * c + (pieces > 0), "CTA %d: slot %d of piece %d", c, x.slot, pieces);
                // a unit's first partial is named by its join, the others are their CTAs' first
                if (x.t0 > 0) CHECK(x.slot == 2 * c && open > 0 && c == join.first / 2 + open, "CTA %d: piece %d", c, open);
                if (x.t0 == 0) {
                    join = walk.join_of(x);
                    const int sub = h % p.subs, h0 = h / p.subs;
                    CHECK(join.first == x.slot && join.row == q.row0 + x.first && join.head == h0 * p.G + sub * p.heads, "CTA %d", c);
                    CHECK(join.heads == (p.G - sub * p.heads < p.heads ? p.G - sub * p.heads : p.heads) && join.lines == n * p.heads, "CTA %d", c);
                    open = 0;
                }
                ++open;
                if (x.t1 == x.tiles) CHECK(join.pieces == open, "CTA %d: %d pieces, not %d", c, join.pieces, open);
            }
            ++pieces;
            done = x.t1;
            if (done == x.tiles) {
                done = 0;
                if (++h == p.H * p.subs) {
                    h = 0;
                    if (x.first + n == q.rows) b = 0, ++r, skip();
                    else ++b;
                }
            }
        }
    }
    CHECK(r == R && expected == total, "%lld of %lld", expected, total);
    CHECK(total == 0 || most - least_places <= 1, "shares of %lld and %lld", least_places, most);
    printf("%lld", total);
    return 0;
}
"""


def cut(tmp_path, kind, H, G, masked, grid, requests):
    exe = tmp_path / "cut"
    args = [kind, H, G, int(masked), grid, len(requests), *(x for q in requests for x in q)]
    if exe.exists():
        r = subprocess.run([str(exe), *map(str, args)], capture_output=True, text=True)
    else:
        r = run(tmp_path, CUT, *args)
    assert r.returncode == 0, (args, r.stdout + r.stderr)
    return int(r.stdout)


GRIDS = {0: (152, 608, 1216), 1: (152,), 2: (152,), 3: (152,)}


def test_cut_gives_every_tile_to_one_cta(tmp_path):
    import random
    rng = random.Random(4)
    for _ in range(120):
        kind = rng.randrange(4)
        G = rng.choice([1, 2, 3, 4, 7, 8, 16] + ([17, 40] if kind < 2 else [128]))
        R = rng.choice([1, 2, 5, 40])
        most = rng.choice([1, 9, 64, 300])
        requests = [(rng.randint(0, rng.choice([1, 100, 5000, 200000])), rng.randint(0, most)) for _ in range(R)]
        masked = rng.random() < 0.4
        if masked:
            requests = [(a, min(n, 256)) for a, n in requests]
        cut(tmp_path, kind, rng.choice([1, 2, 8]), G, masked, rng.choice(GRIDS[kind] + (1, 7)), requests)


@pytest.mark.parametrize("kind,H,G,requests", [
    (0, 8, 16, [(0, 131072)]),                       # one long prompt in units of a row
    (0, 8, 32, [(0, 32768)] * 8),
    (1, 8, 16, [(0, 131072)] * 2),
    (2, 8, 128, [(0, 120000), (5, 1), (0, 120000)]),
    (3, 2, 128, [(1 << 20, 200000)]),
    (2, 43, 1, [(0x7fffff00 - 1, 1)]),               # caches that end where a table may
    (0, 64, 1, [(0x7fffff00 - 1, 1)]),
    (1, 3, 1, [(0x7fffff00 - 300, 300)] * 30),
    (0, 1, 1, [(0, 0), (0x7fffff00 - 7, 7), (0, 0)] * 40),
    (2, 8, 1, [(0x7fffff00 - 1, 1)] * 400),          # shares of 2^30 places, the most there are
    (1, 4, 4, [(0, 4000000)])])
def test_cut_beyond_32_bits_of_places(tmp_path, kind, H, G, requests):
    assert cut(tmp_path, kind, H, G, False, GRIDS[kind][0], requests) > 0x7fffffff
