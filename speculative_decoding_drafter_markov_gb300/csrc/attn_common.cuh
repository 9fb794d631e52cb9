// attn_common.cuh -- what the attention's kernels share: the parameters of a launch,
// the requests of a call and the CTA's share of the work (how it is cut: attn_cut.h).
#pragma once

#include "attn_cut.h"
#include "common.cuh"
#include "target.h"

namespace dspark {
namespace attn {

struct Params : Cut {
    dspark_tree_attention_args a;
    Div page;         // tokens of a page
    int stride;       // floats of a partial's line
    int mixed;        // partials in the order of the tensor-core fragments (see `plain_column`)
    int vec;          // CUDA-core kernel: 16-byte loads are possible
    float scale_log2; // scale * log2(e)
    float *part_o;    // [2 grid][lines][stride]  unnormalised sums
    float2 *part_ml;  // [2 grid][lines]          (maximum of s log2(e), sum of weights)
    Join *join;       // [grid]                   the unit that starts in this CTA and ends in a later one

    __device__ __forceinline__ Request request(int r, bool report = false) const {
        const int row0 = a.row_start[r], row1 = a.row_start[r + 1], len = a.len[r];
        if (row0 == row1) return Request{row0, 0, len};
        const bool ok = row0 >= 0 && row1 > row0 && row1 <= a.N && len >= 0 && (!a.mask || row1 - row0 <= 64 * a.W) &&
                        (long long)len + (row1 - row0) <= (long long)a.max_pages * a.page;
        if (!ok && report) set_err(a.err, DSPARK_ERR_RANGE);
        return Request{row0, ok ? row1 - row0 : 0, len};
    }
};

// Column of place d of a partial's line.  A tensor-core fragment gives a lane the
// columns 8 k + 2 (lane % 4) + {0, 1}; two of them stand side by side, so that the
// four lanes of a row write 64 bytes in one piece.
__device__ __forceinline__ int plain_column(int d) {
    const int in16 = d & 15, pair = (in16 >> 1) & 1;
    return (d & ~15) + 8 * pair + 2 * (in16 >> 2) + (d & 1);
}

// The CTA's share, found by one warp (all its lanes come here and get it): a run of
// requests per lane, no barrier.
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
    for (int r = r0; r < r1; ++r) mine = add_places(mine, request_places(p, p.request(r, blockIdx.x == 0)));
    long long inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc = add_places(inc, y);
    }
    long long total = __shfl_sync(0xffffffffu, inc, 31);
    if (total > (long long)gridDim.x * kMostShare) {
        if (lane == 0 && blockIdx.x == 0) set_err(p.a.err, DSPARK_ERR_UNSUPPORTED);
        total = 0;
    }
    Share s = share_places(p, total, blockIdx.x, gridDim.x);
    if (s.n == 0) return s;
    long long begin = inc - mine;
    int r = r0;
    const bool here = begin <= s.lo && s.lo < begin + mine;
    if (here)
        for (; r1 - r > 1; ++r) {
            const long long n = request_places(p, p.request(r));
            if (s.lo < begin + n) break;
            begin += n;
        }
    const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    s.r = __shfl_sync(0xffffffffu, r, from);
    s.r_begin = __shfl_sync(0xffffffffu, begin, from);
    return s;
}

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
