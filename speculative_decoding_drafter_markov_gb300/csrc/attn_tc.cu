// attn_tc.cu -- attention of drafted rows over a paged cache on the 5th-generation
// tensor cores (bf16, D a multiple of 8 up to 128, pages of a multiple of 8 tokens).
//
// A unit's lines (rows x query heads of a group) fill one or two 128-row MMA
// operands.  Per operand and tile of 128 tokens:
//     S = Q K^T   (Q, K in shared memory, S in tensor memory, fp32)
//     P = 2^(S scale log2(e) - m)   rounded to bf16 over S's columns
//     O += P V    (P in tensor memory, V in shared memory as the MN-major operand)
// Two streams, each with its own S and O and four softmax warps, run side by side:
// with two operands a stream per operand, both over every tile; with one, the
// streams take the even and the odd tiles and are added at the end like two
// partials.  The softmax works and hands P over in halves, so that the first half's
// product runs while the second half is formed.  The maximum m is only moved, and O
// rescaled in tensor memory, when a half exceeds it by 2^8 (any reference gives
// the same result; P stays below 2^8 and the fp32 sums far from overflow): the
// running-maximum softmax of Milakov and Gimelshein (arXiv 1805.02867) with a
// reference that may lag behind.
//
// P is rounded to one bf16 term (the MMA wants A in the type of B, the values): against
// 64 bits the outputs are off by 0.0022 to 0.0023 of their size, the rounding of the output
// alone by 0.0017.  A second term, the rest of P in the half of S's columns that the first
// leaves free, brings that to 0.0017, but doubles the second product and a third of
// the softmax, both in the chain that bounds a tile: 64 caches of up to 8192 tokens 146
// instead of 126 us, 16 of up to 16384 with trees of up to 64 rows 126 instead of 98, 8 of
// up to 131072 with up to 256 lines 587 instead of 433, and with 68 lines 433 instead of 420.
//
// Warps 0-7 softmax, 8 and 10 copy keys and values by TMA, a box per page piece,
// through one ring of slots in the order of their use, 9 copies Q and issues the
// MMAs, 11 walks the CTA's share of the work and hands out its pieces.
//
// Bound by HBM while lines are few: a tile of D = 128 is 64 KB, 2,900 clocks of an
// SM's share of the bandwidth, against 1,030 of MMA per operand.  8 heads of 128, bf16:
// 8 caches of up to 131072 tokens with up to 68 lines take 424 us (6.8 TB/s), 64 of up to
// 8192 with up to 36 lines 127 us (5.6 TB/s, the rest starts and ends of pieces), one row
// over 2047 tokens 12.5 us (latency).  With many lines by the chain from S through the
// softmax to P: 8 caches of up to 131072 with up to 256 lines 435 us, 0.88 PFLOP/s.
// S in half tiles of 64 tokens, to give the softmax its first half earlier, took 4 % more
// than whole tiles: an MMA of 64 columns takes 55 clocks, one of 128 takes 64.
#include "attn_tc_kernel.cuh"

namespace dspark {
namespace attn {

namespace {

// a map of the cache as [n_pages H][page][D], boxes of 64 columns x box tokens
bool encode_cache(CUtensorMap *m, const void *base, const dspark_tree_attention_args &a, int box) {
    const uint64_t dims[3] = {(uint64_t)a.D, (uint64_t)a.page, (uint64_t)a.n_pages * a.H};
    const uint64_t strides[2] = {(uint64_t)a.D * 2, (uint64_t)a.page * a.D * 2};
    const uint32_t bx[3] = {64, (uint32_t)box, 1};
    return encode_bf16_map3(m, base, dims, strides, bx);
}

}  // namespace

bool tc_supported(const dspark_tree_attention_args &a) {
    auto al16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    return a.dtype == DSPARK_BF16 && a.scale >= 0.f && a.D % 8 == 0 && a.D <= 128 && a.page % 8 == 0 && a.Hq / a.H <= 128 && al16(a.q) &&
           al16(a.k_cache) && al16(a.v_cache) && al16(a.out) && a.q_row % 8 == 0 && a.q_head % 8 == 0 && a.q_row > 0 &&
           a.q_head > 0 && a.q_row < (1ll << 38) && a.q_head < (1ll << 38) && tc_available();
}

// One operand while the host's hint says that a request's lines fit it, else two: a unit
// of two reads its keys once for twice the lines.  (8 caches of up to 131072 tokens, up
// to 256 lines: 435 us with two, 572 with one; 4 prompts of up to 4096 rows: 192 and 229;
// 16 caches of up to 1000 tokens, where there are few pieces to share: 33 and 29.)
void tc_shape(const dspark_tree_attention_args &a, int *block_rows, int *lines, int *stride) {
    const int G = a.Hq / a.H, one = 128 / G;
    *block_rows = a.max_rows > one ? 2 * one : one;
    *lines = *block_rows * G;
    *stride = a.D > 64 ? 128 : 64;
}

cudaError_t launch_tc(const Params &p, int grid, cudaStream_t s) {
    TcParams tp{};
    CUtensorMap q, k, v;
    const dspark_tree_attention_args &a = p.a;
    if (!tc_params(tp, p, grid, &q) || !encode_cache(&k, a.k_cache, a, tp.box) || !encode_cache(&v, a.v_cache, a, tp.box))
        return cudaErrorInvalidValue;
    const bool two = p.block_rows > tp.op_rows;
    if (a.D > 64)
        return two ? launch_tc_as<Shape<128, 2>>(tp, grid, q, k, v, s) : launch_tc_as<Shape<128, 1>>(tp, grid, q, k, v, s);
    return two ? launch_tc_as<Shape<64, 2>>(tp, grid, q, k, v, s) : launch_tc_as<Shape<64, 1>>(tp, grid, q, k, v, s);
}

}  // namespace attn
}  // namespace dspark
