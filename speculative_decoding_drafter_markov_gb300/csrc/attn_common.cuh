// attn_common.cuh -- how the attention of drafted rows is cut into work, and how
// the pieces of a row are joined.
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
#pragma once

#include "attn_cut.h"
#include "common.cuh"
#include "target.h"

namespace dspark {
namespace attn {

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
    __device__ __forceinline__ int of(int x) const { return (int)(((unsigned long long)(unsigned)x * mul) >> shift); }
};
inline Div div_by(unsigned by) {
    int l = 0;
    while ((1ull << l) < by) ++l;
    return Div{by, (unsigned)(((1ull << (31 + l)) + by - 1) / by), 31 + l};
}

struct Params {
    dspark_tree_attention_args a;
    int G;            // query heads per key-value head
    int heads;        // of them in a unit: G, or fewer where a unit has not the lines
    int subs;         // units that a group is cut into: ceil(G / heads)
    int block_rows;   // rows of a unit
    int lines;        // block_rows * heads
    int tile_log2;    // tokens of a tile
    int unit_cost;    // empty tiles of a unit before its tiles
    int small_rows;   // a unit of up to so many rows has tiles of small_places,
    Div small_places, large_places;  // one of more rows of large_places
    Div page, ctas;   // tokens of a page; CTAs of the launch
    int stride;       // floats of a partial's line
    int mixed;        // partials in the order of the tensor-core fragments (see `plain_column`)
    int vec;          // CUDA-core kernel: 16-byte loads are possible
    float scale_log2; // scale * log2(e)
    float *part_o;    // [2 grid][lines][stride]  unnormalised sums
    float2 *part_ml;  // [2 grid][lines]          (maximum of s log2(e), sum of weights)
    Join *join;       // [grid]                   the unit that starts in this CTA and ends in a later one
};

// Column of place d of a partial's line.  A tensor-core fragment gives a lane the
// columns 8 k + 2 (lane % 4) + {0, 1}; two of them stand side by side, so that the
// four lanes of a row write 64 bytes in one piece.
__device__ __forceinline__ int plain_column(int d) {
    const int in16 = d & 15, pair = (in16 >> 1) & 1;
    return (d & ~15) + 8 * pair + 2 * (in16 >> 2) + (d & 1);
}

// a request's place: zero rows where its sizes are not usable
struct Request {
    int row0, rows, len;
};

__device__ __forceinline__ Request request_of(const Params &p, int r, bool report) {
    const dspark_tree_attention_args &a = p.a;
    const int row0 = a.row_start[r], row1 = a.row_start[r + 1], len = a.len[r];
    if (row0 == row1) return Request{row0, 0, len};
    const bool ok = row0 >= 0 && row1 > row0 && row1 <= a.N && len >= 0 && (!a.mask || row1 - row0 <= 64 * a.W) &&
                    (long long)len + (row1 - row0) <= (long long)a.max_pages * a.page;
    if (!ok && report) set_err(a.err, DSPARK_ERR_RANGE);
    return Request{row0, ok ? row1 - row0 : 0, len};
}

__device__ __forceinline__ Request request_of(const Params &p, int r) { return request_of(p, r, false); }

__device__ __forceinline__ int blocks_of(const Params &p, int rows) {
    return rows <= p.block_rows ? (rows > 0 ? 1 : 0) : (rows + p.block_rows - 1) / p.block_rows;
}

// tokens that the rows of block b can see
__device__ __forceinline__ int tokens_of(const Params &p, const Request &q, int b) {
    return q.len + (p.a.mask ? q.rows : min(q.rows, (b + 1) * p.block_rows));
}

__device__ __forceinline__ int tiles_of(const Params &p, const Request &q, int b) {
    return (int)(((unsigned)tokens_of(p, q, b) + (1u << p.tile_log2) - 1) >> p.tile_log2);
}

// places of a tile of block b
__device__ __forceinline__ const Div &tile_places(const Params &p, const Request &q, int b) {
    return min(p.block_rows, q.rows - b * p.block_rows) > p.small_rows ? p.large_places : p.small_places;
}

__device__ __forceinline__ long long request_places(const Params &p, const Request &q) {
    const int n = blocks_of(p, q.rows);
    long long t = 0;
    for (int b = 0; b < n; ++b) t += (long long)(tiles_of(p, q, b) + p.unit_cost) * tile_places(p, q, b).by;
    return t * (p.a.H * p.subs);
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

// The CTA's share of the line and the place where it starts, found by one warp (all
// its lanes come here and get it): a run of requests per lane, no barrier.
struct Share {
    int lo, hi;
    int each, more;      // places of a CTA's share; the first `more` CTAs have one more
    int r;               // request of place lo
    int r_begin;         // its first place
};

__device__ inline Share share_of(const Params &p) {
    const int lane = threadIdx.x & 31, R = p.a.R;
    const int per = (R + 31) / 32, r0 = min(R, lane * per), r1 = min(R, r0 + per);
    long long mine = 0;
    // (little code: it comes from L2 at the start of a launch, and is run once)
#pragma unroll 1
    for (int r = r0 + 1; r < r1; ++r) {
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.a.row_start + r + 1));
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p.a.len + r));
    }
#pragma unroll 1
    for (int r = r0; r < r1; ++r) mine += request_places(p, request_of(p, r, blockIdx.x == 0));
    long long inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
    }
    long long total = __shfl_sync(0xffffffffu, inc, 31);
    Share s{0, 0, 1, 0, 0, 0};
    if (total > 0x7fffffffll) {  // far above the work of a call: not counted in 64 bits
        if (lane == 0 && blockIdx.x == 0) set_err(p.a.err, DSPARK_ERR_UNSUPPORTED);
        total = 0;
    }
    // no share is smaller than a tile, so every CTA between a unit's first and last one
    // has a tile of it
    const unsigned t = (unsigned)total, c = blockIdx.x, ctas = min(gridDim.x, (unsigned)max(1, p.large_places.of(t)));
    if (t == 0 || c >= ctas) return s;
    s.each = ctas == p.ctas.by ? p.ctas.of(t) : t / ctas;
    s.more = t - s.each * ctas;
    s.lo = c * s.each + min((int)c, s.more);
    s.hi = s.lo + s.each + ((int)c < s.more ? 1 : 0);
    int begin = (int)(inc - mine), r = r0;
    const bool here = begin <= s.lo && s.lo < begin + (int)mine;
    if (here)
        for (; r1 - r0 > 1; ++r) {
            const int n = (int)request_places(p, request_of(p, r));
            if (s.lo < begin + n) break;
            begin += n;
        }
    const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    s.r = __shfl_sync(0xffffffffu, r, from);
    s.r_begin = __shfl_sync(0xffffffffu, begin, from);
    return s;
}

// Walks the pieces of a CTA's share in order.
struct Walk {
    const Params &p;
    Share s;
    int at;            // next place of the line
    int r, b, h;       // its unit
    int begin;         // the unit's first place
    int tiles;         // of the unit
    Div places;        // of one of its tiles
    int blocks;        // of the request
    Request q;
    bool first;

    __device__ __forceinline__ Walk(const Params &p_, const Share &s_) : p(p_), s(s_), at(s_.lo), b(0), h(0), first(true) {
        if (s.lo >= s.hi) return;
        r = s.r;
        q = request_of(p, r);
        blocks = blocks_of(p, q.rows);
        int left = s.lo - s.r_begin;
        for (;; ++b) {
            shape();
            const int line = (tiles + p.unit_cost) * places.by * p.a.H * p.subs;
            if (left < line) break;
            left -= line;
        }
        const int unit = (tiles + p.unit_cost) * places.by;
        h = (unsigned)left / (unsigned)unit;
        begin = s.lo - (left - h * unit);
    }

    __device__ __forceinline__ void shape() {
        tiles = tiles_of(p, q, b);
        places = tile_places(p, q, b);
    }

    // the unit's first tile at or after a place of the line
    __device__ __forceinline__ int tile_at(int place) const {
        const int d = place - (begin + p.unit_cost * (int)places.by);
        return d <= 0 ? 0 : min(tiles, places.of(d + (int)places.by - 1));
    }

    __device__ __forceinline__ bool next(Piece &out) {
        if (at >= s.hi) return false;
        out.t0 = tile_at(at);
        if (out.t0 == tiles) {  // the share begins within the unit's last tile
            advance();
            if (at >= s.hi) return false;
            out.t0 = 0;
        }
        out.t1 = tile_at(s.hi);
        if (out.t0 >= out.t1) return false;  // the unit's first tile is another CTA's
        out.r = r;
        out.head = h;
        out.tiles = tiles;
        out.row0 = q.row0;
        out.rows = q.rows;
        out.len = q.len;
        out.first = b * p.block_rows;
        out.n = min(p.block_rows, q.rows - out.first);
        out.tokens = tokens_of(p, q, b);
        out.slot = out.t0 == 0 && out.t1 == tiles ? -1 : 2 * (int)blockIdx.x + (first ? 0 : 1);
        first = false;
        if (out.t1 == tiles) advance();
        else at = s.hi;
        return true;
    }

    // the unit is done: the next head, block or request, if its places begin in the share
    __device__ __forceinline__ void advance() {
        at = begin + (p.unit_cost + tiles) * (int)places.by;
        if (at >= s.hi) return;
        begin = at;
        if (++h < p.a.H * p.subs) return;
        h = 0;
        if (++b == blocks) {
            b = 0;
            do {
                q = request_of(p, ++r);
            } while (q.rows == 0);
            blocks = blocks_of(p, q.rows);
        }
        shape();
    }

    // what the second launch needs of a piece that starts a unit and does not end it
    // (the last one of its share: the walk still stands at its unit)
    __device__ __forceinline__ Join join_of(const Piece &x) const {
        const unsigned last = begin + (p.unit_cost + x.tiles - 1) * (int)places.by;
        const unsigned big = (unsigned)s.more * (s.each + 1);
        const unsigned c = last < big ? last / (unsigned)(s.each + 1) : s.more + (last - big) / (unsigned)s.each;
        const int sub = p.subs == 1 ? 0 : x.head % p.subs, h0 = p.subs == 1 ? x.head : x.head / p.subs;
        return Join{(int)c - (int)blockIdx.x + 1, x.slot, x.row0 + x.first, h0 * p.G + sub * p.heads,
                    min(p.heads, p.G - sub * p.heads), x.n * p.heads};
    }
};

__device__ __forceinline__ void store_out(const Params &p, size_t at, float v) {
    if (p.a.dtype == DSPARK_BF16) static_cast<__nv_bfloat16 *>(p.a.out)[at] = __float2bfloat16_rn(v);
    else static_cast<float *>(p.a.out)[at] = v;
}

// ln of the sum of exponentials from the maximum of s log2(e) and the weights' sum
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.f ? (m + __log2f(l)) * kLn2 : (l == l ? -INFINITY : l); }

size_t workspace_bytes(int grid, int lines, int stride);
void carve(Params &p, void *ws, int grid);
// the tensor-core kernel: one CTA per SM
bool tc_supported(const dspark_tree_attention_args &a);
void tc_shape(const dspark_tree_attention_args &a, int *block_rows, int *lines, int *stride);
cudaError_t launch_tc(Params p, int grid, cudaStream_t s);
// the fp32 kernel: units of kSimtLines lines, as the general CUDA-core kernel
constexpr int kSimtLines = 16;
bool f32_supported(const dspark_tree_attention_args &a);
int f32_grid();
cudaError_t launch_f32(Params p, int grid, cudaStream_t s);
cudaError_t launch_join(const Params &p, int grid, cudaStream_t s);

}  // namespace attn
}  // namespace dspark
