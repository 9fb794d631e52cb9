// attn4_tc.cu -- the tensor-core attention over a cache in 4 bits.
//
// The kernel of attn_tc.cu with a step between the copies and the products: packed tiles come into
// rings of their own by bulk copies, codes and scales of a page piece apart, and warps beside the
// others unpack them into the ring that the MMAs read (unpack_tiles), keys and values apart.
// Scores are products of bf16 numbers, weights and values of fp16 ones.
//
// 8 caches of up to 131072 tokens, up to 17 rows of 4 query heads (810 MB, 79 GFLOP): 446 us, as long as over 16-bit
// caches (419) of 3.6 times the bytes; 16 trees of up to 64 rows over up to 16384 tokens: 140 us (97).
// What bounds it is the chain of a tile: keys unpacked and visible to the tensor cores (700 clocks of work and
// 1300 until the fence has passed), S, its softmax (3200 clocks for 128 x 128 with the other roles beside it), the
// second product.  Over a quarter of the first case's tokens the tensor pipe works for 38 % of the time and half of the
// issue slots are used, by waits too.  Every shape spills: 40 to 44 bytes of stores and 48 to 76 of loads a thread at 128
// registers (one operand) or 96 (two).  Head sizes between 64 and 128 run as 128.
#include "attn_tc_kernel.cuh"

namespace dspark {
namespace attn {

bool tc4_supported(const dspark_tree_attention_args &a) {
    auto al16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    int box = a.page & -a.page;  // tokens of a copy
    if (box > kTile) box = kTile;
    return a.dtype == DSPARK_BF16 && a.scale >= 0.f && a.D <= 128 && box >= 8 && box * a.D % 256 == 0 && a.Hq / a.H <= 128 && al16(a.q) &&
           al16(a.out) && a.q_row % 8 == 0 && a.q_head % 8 == 0 && a.q_row > 0 && a.q_head > 0 && a.q_row < (1ll << 38) &&
           a.q_head < (1ll << 38) && tc_available();
}

cudaError_t launch_tc4(const Params &p, int grid, cudaStream_t s) {
    TcParams tp{};
    CUtensorMap q;
    if (!tc_params(tp, p, grid, &q)) return cudaErrorInvalidValue;
    const bool two = p.block_rows > tp.op_rows;
    if (p.a.D > 64)
        return two ? launch_tc_as<Shape<128, 2, true>>(tp, grid, q, q, q, s) : launch_tc_as<Shape<128, 1, true>>(tp, grid, q, q, q, s);
    return two ? launch_tc_as<Shape<64, 2, true>>(tp, grid, q, q, q, s) : launch_tc_as<Shape<64, 1, true>>(tp, grid, q, q, q, s);
}

}  // namespace attn
}  // namespace dspark
