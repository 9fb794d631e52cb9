// attn_cut.h -- how the attention of drafted rows is cut into work.  Arithmetic alone,
// which any C++ compiler takes, so that the CPU can walk it to the ends of its ranges.
//
// A unit is one key-value head of one request and a block of its rows: every
// row with every query head of the group that shares the keys (row jj of the
// block and head g of the group in line jj heads + g).  Its tokens are walked in
// tiles.  The tiles of all units stand in one line -- by request, block, head --
// and each CTA takes an equal, consecutive share of the line, whatever the
// lengths of the requests are: a long cache is spread over many CTAs, many short
// ones are packed into one, and no length reaches the host.  A tile has as many places
// in the line as its time is worth, and before its tiles a unit has `unit_cost` empty
// tiles' worth of places for its start and end, so that CTAs with many short units get
// fewer tiles.  A tile is the CTA's whose share holds its first place.  A CTA leaves a unit
// that it did not do whole as a partial (unnormalised sums, maximum and sum of
// the weights); a second launch joins the partials of each unit.
//
// The line is counted in 64 bits: its places grow with the square of a prompt's rows
// (131072 rows in units of one row, tiles of 32 tokens, 8 heads: 2.1e9).  A CTA's share
// and a unit fit 32 bits, and a CTA counts from the start of its share.
#pragma once

#ifdef __CUDACC__
#define DSPARK_CUT __device__ __forceinline__
#else
#define DSPARK_CUT inline
#endif

namespace dspark {
namespace attn {

DSPARK_CUT int least(int a, int b) { return a < b ? a : b; }

// The token by which a copying lane finds its page: the first of box b (of `box`
// tokens) of tile t.  There are lanes for more boxes than a tile has: those look where
// its last box does, so that no token number passes the end of the tile, the only one
// that is known to fit 32 bits; nor does any pass the unit's last token.
DSPARK_CUT int lookup_token(int t, int tile_log2, int b, int box, int last) {
    return least((t << tile_log2) + least(b * box, (1 << tile_log2) - box), last);
}

struct Join {
    int pieces;       // 0: none
    int first;        // its first partial; the others are the first partials of the next CTAs
    int row, head, heads, lines;
};

// Division of a number below 2^31 by one that the host knows, as a product and a shift:
// the divide routine's chain is long where one thread prepares a CTA's work.  With
// 2^(l - 1) < by <= 2^l and mul = ceil(2^(31 + l) / by), x mul / 2^(31 + l) is above
// x / by by less than 1 / by.
struct Div {
    unsigned by, mul;
    int shift;
    DSPARK_CUT int of(int x) const { return (int)(((unsigned long long)(unsigned)x * mul) >> shift); }
};
inline Div div_by(unsigned by) {
    int l = 0;
    while ((1ull << l) < by) ++l;
    return Div{by, (unsigned)(((1ull << (31 + l)) + by - 1) / by), 31 + l};
}

// x / by, which fits 32 bits: by the short routine where x does too, else bit by bit (the
// routine for 64 bits, though never called, took the fp32 kernel from 95 to 98.5 us for
// 16 caches of up to 8192 tokens)
DSPARK_CUT unsigned quotient(unsigned long long x, unsigned by) {
    if ((x >> 32) == 0) return (unsigned)x / by;
    unsigned q = 0;
#ifdef __CUDACC__
#pragma unroll 1
#endif
    for (int i = 31; i >= 0; --i)
        if ((x >> i) >= by) {
            x -= (unsigned long long)by << i;
            q |= 1u << i;
        }
    return q;
}

struct Cut {
    int H;            // key-value heads
    int G;            // query heads per key-value head
    int heads;        // of them in a unit: G, or fewer where a unit has not the lines
    int subs;         // units that a group is cut into: ceil(G / heads)
    int block_rows;   // rows of a unit
    int lines;        // block_rows * heads
    int tile_log2;    // tokens of a tile
    int unit_cost;    // empty tiles of a unit before its tiles
    int small_rows;   // a unit of up to so many rows has tiles of small_places,
    Div small_places, large_places;  // one of more rows of large_places
    Div ctas;         // CTAs of the launch
    int masked;       // rows see by masks: a unit's tokens are all of the request's
};

// a request's place: zero rows where its sizes are not usable
struct Request {
    int row0, rows, len;
};

DSPARK_CUT int blocks_of(const Cut &p, int rows) {
    return rows <= p.block_rows ? (rows > 0 ? 1 : 0) : (rows - 1) / p.block_rows + 1;
}

// tokens that the rows of block b can see
DSPARK_CUT int tokens_of(const Cut &p, const Request &q, int b) {
    const int left = q.rows - b * p.block_rows;  // rows of the request from block b on
    return q.len + (p.masked || left <= p.block_rows ? q.rows : (b + 1) * p.block_rows);
}

DSPARK_CUT int tiles_of(const Cut &p, const Request &q, int b) {
    return (int)(((unsigned)tokens_of(p, q, b) + (1u << p.tile_log2) - 1) >> p.tile_log2);
}

// places of a tile of block b
DSPARK_CUT const Div &tile_places(const Cut &p, const Request &q, int b) {
    return least(p.block_rows, q.rows - b * p.block_rows) > p.small_rows ? p.large_places : p.small_places;
}

// A request has at most N Hq < 2^31 units of less than 2^27 places, and so have all
// requests together unless their rows overlap: sums stop here, where no call's line ends.
constexpr long long kMostPlaces = 1ll << 58;

DSPARK_CUT long long add_places(long long a, long long b) { return a + b < kMostPlaces ? a + b : kMostPlaces; }

DSPARK_CUT long long request_places(const Cut &p, const Request &q) {
    const int n = blocks_of(p, q.rows);
    long long t = 0;
    for (int b = 0; b < n; ++b) t += (long long)(tiles_of(p, q, b) + p.unit_cost) * tile_places(p, q, b).by;
    return t * (p.H * p.subs);
}

// One CTA's piece of a unit.
struct Piece {
    int r, head;     // request; unit's place among the request's heads: h subs + sub
    int t0, t1;      // its tiles
    int tiles;       // the unit's tiles
    int row0;        // the request's first row
    int rows, len;   // of the request
    int first, n;    // the unit's rows: first row and how many
    int tokens;      // the unit's tokens
    int slot;        // partial to leave it in, or -1: the unit is whole
};

// The most places of a CTA's share: minutes of work.
constexpr int kMostShare = 1 << 30;

// A CTA's share of the line and the place where it starts.
struct Share {
    long long lo;        // its first place
    int n;               // how many
    int each, more;      // places of any CTA's share; the first `more` CTAs have one more
    int cta;
    int r;               // request of place lo
    long long r_begin;   // its first place
};

// CTA `cta` of `grid`: its places of `total`.  No share is smaller than a tile, so every
// CTA between a unit's first and last one has a tile of it.
DSPARK_CUT Share share_places(const Cut &p, long long total, int cta, int grid) {
    Share s{0, 0, 1, 0, cta, 0, 0};
    const int by = (int)p.large_places.by;
    const int ctas = total >= (long long)grid * by ? grid : total < by ? 1 : p.large_places.of((int)total);
    if (total == 0 || cta >= ctas) return s;
    s.each = (total >> 31) == 0 && ctas == (int)p.ctas.by ? p.ctas.of((int)total) : (int)quotient(total, (unsigned)ctas);
    s.more = (int)(total - (long long)s.each * ctas);
    s.lo = (long long)cta * s.each + least(cta, s.more);
    s.n = s.each + (cta < s.more ? 1 : 0);
    return s;
}

// Walks the pieces of a CTA's share in order; places are counted from the share's first.
// P: a Cut with `request(r)`.
template <typename P>
struct Walk {
    const P &p;
    int n, each, more, cta;  // of the share
    int at;            // next place
    int r, b, h;       // its unit
    int begin;         // the unit's first place
    int tiles;         // of the unit
    Div places;        // of one of its tiles
    int blocks;        // of the request
    Request q;
    bool first;

    DSPARK_CUT Walk(const P &p_, const Share &s) : p(p_), n(s.n), each(s.each), more(s.more), cta(s.cta), at(0), b(0), h(0), first(true) {
        if (n == 0) return;
        r = s.r;
        q = p.request(r);
        blocks = blocks_of(p, q.rows);
        long long left = s.lo - s.r_begin;
        for (;; ++b) {
            shape();
            const long long line = (long long)unit_places() * (p.H * p.subs);
            if (left < line) break;
            left -= line;
        }
        h = (int)quotient(left, (unsigned)unit_places());
        begin = (int)((long long)h * unit_places() - left);
    }

    DSPARK_CUT void shape() {
        tiles = tiles_of(p, q, b);
        places = tile_places(p, q, b);
    }

    DSPARK_CUT int unit_places() const { return (tiles + p.unit_cost) * (int)places.by; }

    // the unit's first tile at or after a place
    DSPARK_CUT int tile_at(int place) const {
        const int d = place - (begin + p.unit_cost * (int)places.by);
        return d <= 0 ? 0 : least(tiles, places.of(d + (int)places.by - 1));
    }

    DSPARK_CUT bool next(Piece &out) {
        if (at >= n) return false;
        out.t0 = tile_at(at);
        if (out.t0 == tiles) {  // the share begins within the unit's last tile
            advance();
            if (at >= n) return false;
            out.t0 = 0;
        }
        out.t1 = tile_at(n);
        if (out.t0 >= out.t1) return false;  // the unit's first tile is another CTA's
        out.r = r;
        out.head = h;
        out.tiles = tiles;
        out.row0 = q.row0;
        out.rows = q.rows;
        out.len = q.len;
        out.first = b * p.block_rows;
        out.n = least(p.block_rows, q.rows - out.first);
        out.tokens = tokens_of(p, q, b);
        out.slot = out.t0 == 0 && out.t1 == tiles ? -1 : 2 * cta + (first ? 0 : 1);
        first = false;
        if (out.t1 == tiles) advance();
        else at = n;
        return true;
    }

    // the unit is done: the next head, block or request, if its places begin in the share
    DSPARK_CUT void advance() {
        at = begin + unit_places();
        if (at >= n) return;
        begin = at;
        if (++h < p.H * p.subs) return;
        h = 0;
        if (++b == blocks) {
            b = 0;
            do {
                q = p.request(++r);
            } while (q.rows == 0);
            blocks = blocks_of(p, q.rows);
        }
        shape();
    }

    // what the second launch needs of a piece that starts a unit and does not end it
    // (the last one of its share: the walk still stands at its unit)
    DSPARK_CUT Join join_of(const Piece &x) const {
        const int last = begin + unit_places() - (int)places.by;  // the last tile's first place
        const int long_ones = more > cta ? more - cta : 0;         // CTAs from this one on with a place more
        const long long big = (long long)long_ones * (each + 1);
        // CTAs after this one
        const int c = last < big ? (unsigned)last / (unsigned)(each + 1) : long_ones + (unsigned)(last - big) / (unsigned)each;
        const int sub = p.subs == 1 ? 0 : x.head % p.subs, h0 = p.subs == 1 ? x.head : x.head / p.subs;
        return Join{c + 1, x.slot, x.row0 + x.first, h0 * p.G + sub * p.heads, least(p.heads, p.G - sub * p.heads), x.n * p.heads};
    }
};

}  // namespace attn
}  // namespace dspark
