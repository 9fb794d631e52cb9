// attn_common.cuh -- how the attention of drafted rows is cut into work, and how
// the pieces of a row are joined.
//
// A unit is one key-value head of one request and a block of up to `block` of
// its query rows (row j and query head g of the group in line j G + g, so the
// heads that share keys share a unit).  Its tokens are walked in tiles.  The
// tiles of all units stand in one line -- by request, block of rows, head --
// and each CTA takes an equal, consecutive share of the line, whatever the
// lengths of the requests are: a long cache is spread over many CTAs, many
// short ones are packed into one, and no length reaches the host.  A CTA leaves
// a unit that it did not do whole as a partial (unnormalised sums, maximum and
// sum of the weights); a second launch joins the partials of each unit.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace dspark {
namespace attn {

struct Params {
    dspark_tree_attention_args a;
    int G;            // query heads per key-value head
    int block;        // lines of a unit
    int tile;         // tokens of a tile
    int vec;          // CUDA-core kernel: 16-byte loads are possible
    float scale_log2; // scale * log2(e)
    float *part_o;    // [2 grid][block][D]  unnormalised sums
    float2 *part_ml;  // [2 grid][block]     (maximum of s log2(e), sum of weights)
    struct Join *join;  // [grid]            the unit that starts in this CTA and ends in a later one
};

struct Join {
    int pieces;       // 0: none
    int first;        // its first partial; the others are the first partials of the next CTAs
    int row0, h, line0, lines;
};

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

__device__ __forceinline__ int blocks_of(const Params &p, const Request &q) {
    return (q.rows * p.G + p.block - 1) / p.block;
}

// tokens that block b of a request's lines can see
__device__ __forceinline__ int tokens_of(const Params &p, const Request &q, int b) {
    if (p.a.mask) return q.len + q.rows;
    const int last = min(q.rows * p.G, (b + 1) * p.block) - 1;
    return q.len + last / p.G + 1;
}

__device__ __forceinline__ int tiles_of(const Params &p, const Request &q, int b) {
    return (tokens_of(p, q, b) + p.tile - 1) / p.tile;
}

__device__ __forceinline__ long long request_tiles(const Params &p, const Request &q) {
    const int n = blocks_of(p, q);
    long long t = 0;
    for (int b = 0; b < n; ++b) t += tiles_of(p, q, b);
    return t * p.a.H;
}

// One CTA's piece of a unit.
struct Piece {
    int r, b, h;
    int t0, t1;      // its tiles
    int tiles;       // the unit's tiles
    int row0, rows, len;
    int line0, lines;
    int tokens;      // the unit's tokens
    int slot;        // partial to leave it in, or -1: the unit is whole
};

// The CTA's share of the line and the place where it starts.  Every thread of
// the CTA calls this once; `sh` is shared scratch of 2 + 2 (threads / 32) words.
struct Share {
    long long lo, hi, total;
    int ctas;            // CTAs that have a share
    int r;               // request of tile lo
    long long r_begin;   // its first tile
};

__device__ inline Share share_of(const Params &p, long long *sh) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
    const int R = p.a.R, per = (R + (int)blockDim.x - 1) / (int)blockDim.x;
    const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
    long long mine = 0;
    for (int r = r0; r < r1; ++r) mine += request_tiles(p, request_of(p, r, blockIdx.x == 0));
    long long inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
    }
    if (lane == 31) sh[2 + warp] = inc;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < nwarps; ++w) {
        if (w < warp) before += sh[2 + w];
        total += sh[2 + w];
    }
    Share s;
    s.total = total;
    s.ctas = (int)min((long long)gridDim.x, total);
    s.lo = s.hi = 0;
    s.r = 0;
    s.r_begin = 0;
    if ((int)blockIdx.x < s.ctas) {
        s.lo = total * blockIdx.x / s.ctas;
        s.hi = total * (blockIdx.x + 1) / s.ctas;
        long long begin = before + inc - mine;
        if (begin <= s.lo && s.lo < begin + mine) {
            int r = r0;
            for (;;) {
                const long long t = request_tiles(p, request_of(p, r, false));
                if (s.lo < begin + t) break;
                begin += t;
                ++r;
            }
            sh[0] = r;
            sh[1] = begin;
        }
    }
    __syncthreads();
    s.r = (int)sh[0];
    s.r_begin = sh[1];
    return s;
}

// Walks the pieces of a CTA's share in order.
struct Walk {
    const Params &p;
    Share s;
    long long at;      // next tile of the line
    int r, b, h, t;    // its place
    Request q;
    bool first;

    __device__ __forceinline__ Walk(const Params &p_, const Share &s_) : p(p_), s(s_), at(s_.lo), b(0), h(0), first(true) {
        if (s.lo >= s.hi) return;
        r = s.r;
        q = request_of(p, r, false);
        long long left = s.lo - s.r_begin;
        for (;; ++b) {
            const long long line = (long long)tiles_of(p, q, b) * p.a.H;
            if (left < line) break;
            left -= line;
        }
        const int tiles = tiles_of(p, q, b);
        h = (int)(left / tiles);
        t = (int)(left % tiles);
    }

    __device__ __forceinline__ bool next(Piece &out) {
        if (at >= s.hi) return false;
        const int tiles = tiles_of(p, q, b);
        out.r = r;
        out.b = b;
        out.h = h;
        out.t0 = t;
        out.t1 = (int)min((long long)tiles, t + (s.hi - at));
        out.tiles = tiles;
        out.row0 = q.row0;
        out.rows = q.rows;
        out.len = q.len;
        out.line0 = b * p.block;
        out.lines = min(p.block, q.rows * p.G - out.line0);
        out.tokens = tokens_of(p, q, b);
        out.slot = out.t0 == 0 && out.t1 == tiles ? -1 : 2 * (int)blockIdx.x + (first ? 0 : 1);
        first = false;
        at += out.t1 - t;
        if (at < s.hi) {  // the unit is done: the next head, block or request
            t = 0;
            if (++h == p.a.H) {
                h = 0;
                if (++b == blocks_of(p, q)) {
                    b = 0;
                    do {
                        q = request_of(p, ++r, false);
                    } while (q.rows == 0);
                }
            }
        }
        return true;
    }

    // what the second launch needs of a piece that starts a unit and does not end it
    __device__ __forceinline__ Join join_of(const Piece &x) const {
        const long long end = s.hi - x.t1 + x.tiles;  // the piece is the share's last one
        int c = blockIdx.x;
        while (s.total * (c + 1) / s.ctas < end) ++c;
        return Join{c - (int)blockIdx.x + 1, x.slot, x.row0, x.h, x.line0, x.lines};
    }
};

__device__ __forceinline__ void store_out(const Params &p, size_t at, float v) {
    if (p.a.dtype == DSPARK_BF16) static_cast<__nv_bfloat16 *>(p.a.out)[at] = __float2bfloat16_rn(v);
    else static_cast<float *>(p.a.out)[at] = v;
}

// ln of the sum of exponentials from the maximum of s log2(e) and the weights' sum
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.f ? (m + __log2f(l)) * kLn2 : (l == l ? -INFINITY : l); }

size_t workspace_bytes(int grid, int block, int D);
void carve(Params &p, void *ws, int grid);
// the tensor-core kernel: one CTA per SM
bool tc_supported(const dspark_tree_attention_args &a);
int tc_block(const dspark_tree_attention_args &a);
cudaError_t launch_tc(Params p, int grid, cudaStream_t s);
cudaError_t launch_join(const Params &p, int grid, cudaStream_t s);

}  // namespace attn
}  // namespace dspark
