// paged.cu -- the paged key-value cache around the target's pass: the batch map
// of a cycle (pages, row starts, slots, positions, ancestor masks) and the
// write of the rows' keys and values.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace dspark {

namespace {

// ---------------------------------------------------------------- batch map
// Three running sums over the requests give everything: rows (row_start), pages
// given back and pages taken.  Every CTA forms them for itself in shared memory
// (R is small: 3 x 4 (R + 1) bytes), so no CTA waits for another and the call is
// one launch however many CTAs fill its outputs.  What makes this race-free:
// * the k-th page taken is the k-th page given back while there are any
//   (k < m: last in, first out), found in the giver's table row, which nobody
//   writes; after that it is entry n_free - 1 - (k - m) of the stack, below
//   every entry that the returns write;
// * table entries are written only at and beyond a taker's held pages, where
//   nobody reads them (a row's slot takes its page by the same rule);
// * held and n_free are not written (their new values go elsewhere).
// Bound by latency: at R = 4 one CTA's chain of a load, a scan and a store.
constexpr int kMapThreads = 512;

struct MapSums {
    int *rows, *less, *more;  // [R + 1] each, exclusive
};

// the last r with sum[r] <= k (sum[R] > k): the request that holds item k
__device__ __forceinline__ int holder(const int *sum, int R, int k) {
    int lo = 0, hi = R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] <= k) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ long long need_of(const dspark_page_map_args &a, int r) {
    return ((long long)a.len[r] + a.rows[r] + a.page - 1) / a.page;
}

__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const dspark_page_map_args a) {
    extern __shared__ int sh[];
    const int R = a.R;
    const MapSums s{sh, sh + (R + 1), sh + 2 * (R + 1)};
    __shared__ long long wsum[3][kMapThreads / 32];
    __shared__ int bad_any;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad_any = 0;

    // a run of consecutive requests per thread, then a scan over the threads
    const int per = (R + kMapThreads - 1) / kMapThreads;
    const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
    long long v[3] = {0, 0, 0};
    bool bad = false;
    for (int r = r0; r < r1; ++r) {
        const long long need = need_of(a, r);
        const int held = a.held[r];
        if (a.len[r] < 0 || a.rows[r] < 0 || held < 0 || held > a.max_pages || need > a.max_pages ||
            (a.mask && a.rows[r] > 64 * a.W))
            bad = true;
        v[0] += a.rows[r];
        if (held > need) v[1] += held - need;
        else v[2] += need - held;
    }
    long long inc[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        long long x = v[i];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        inc[i] = x;
        if (lane == 31) wsum[i][warp] = x;
    }
    __syncthreads();
    if (bad) bad_any = 1;
    long long base[3], total[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        long long b = 0, t = 0;
        for (int w = 0; w < kMapThreads / 32; ++w) {
            const long long x = wsum[i][w];
            if (w < warp) b += x;
            t += x;
        }
        base[i] = b + inc[i] - v[i];
        total[i] = t;
    }
    for (int r = r0; r < r1; ++r) {
        s.rows[r] = (int)base[0];
        s.less[r] = (int)base[1];
        s.more[r] = (int)base[2];
        const long long need = need_of(a, r);
        const int held = a.held[r];
        base[0] += a.rows[r];
        if (held > need) base[1] += held - need;
        else base[2] += need - held;
    }
    if (tid == 0) {
        s.rows[R] = (int)total[0];
        s.less[R] = (int)total[1];
        s.more[R] = (int)total[2];
    }
    __syncthreads();

    const int before = *a.n_free;
    const bool fail = bad_any || total[0] > a.N || (a.parents && total[0] > a.n_parents) || before < 0 ||
                      before + total[1] > a.n_pages || total[2] > before + total[1];
    const int first = blockIdx.x * kMapThreads + tid, step = gridDim.x * kMapThreads;
    if (fail) {
        if (first == 0) {
            set_err(a.err, DSPARK_ERR_RANGE);
            *a.n_free_out = before;
        }
        for (int r = first; r <= R; r += step) {
            a.row_start[r] = 0;
            if (r < R) a.held_out[r] = a.held[r];
        }
        for (int i = first; i < a.N; i += step) {
            a.slot[i] = -1;
            a.pos[i] = 0;
            for (int w = 0; w < (a.mask ? a.W : 0); ++w) a.mask[(size_t)i * a.W + w] = 0;
        }
        return;
    }
    const int m = (int)total[1], taken = (int)total[2], after = before + m;
    auto given = [&](int k) {  // the k-th page given back
        const int r = holder(s.less, R, k);
        return a.table[(size_t)r * a.max_pages + need_of(a, r) + (k - s.less[r])];
    };
    auto page_of = [&](int k) {  // the k-th page taken
        return k < m ? given(k) : a.free_list[before - 1 - (k - m)];
    };

    if (first == 0) *a.n_free_out = after - taken;
    for (int r = first; r <= R; r += step) {
        a.row_start[r] = s.rows[r];
        if (r < R) a.held_out[r] = (int)need_of(a, r);
    }
    for (int k = first; k < m; k += step) a.free_list[after - 1 - k] = given(k);
    for (int k = first; k < taken; k += step) {
        const int r = holder(s.more, R, k);
        a.table[(size_t)r * a.max_pages + a.held[r] + (k - s.more[r])] = page_of(k);
    }
    for (int i = first; i < a.N; i += step) {
        int slot = -1, pos = 0;
        if (i < s.rows[R]) {
            const int r = holder(s.rows, R, i), start = s.rows[r], j = i - start;
            const int t = a.len[r] + j, pi = t / a.page, held = a.held[r];
            const int pg = pi < held ? a.table[(size_t)r * a.max_pages + pi] : page_of(s.more[r] + pi - held);
            slot = pg * a.page + t % a.page;
            pos = t;
            if (a.parents) {
                // walk up: a parent is an earlier row, so the walk ends
                int depth = 0, at = j;
                uint64_t word = 0;
                int w = j >> 6;
                for (;;) {
                    word |= 1ull << (at & 63);
                    int p = a.parents[start + at];
                    if (p >= at) {
                        set_err(a.err, DSPARK_ERR_RANGE);
                        p = -1;
                    }
                    // words are finished from the highest down
                    while (w > (p < 0 ? -1 : p >> 6)) {
                        a.mask[(size_t)i * a.W + w] = word;
                        word = 0;
                        --w;
                    }
                    if (p < 0) break;
                    at = p;
                    ++depth;
                }
                for (int hw = (j >> 6) + 1; hw < a.W; ++hw) a.mask[(size_t)i * a.W + hw] = 0;
                pos = a.len[r] + depth;
            }
        } else if (a.parents) {
            for (int w = 0; w < a.W; ++w) a.mask[(size_t)i * a.W + w] = 0;
        }
        a.slot[i] = slot;
        a.pos[i] = pos;
    }
}

// ---------------------------------------------------------------- cache write
// A copy of 2 N H D elements: bound by HBM (read once, written once).  A CTA
// takes kStoreRows rows, its threads the 16-byte pieces of their keys and
// values in order, so that reads and writes of a head are both adjacent.
constexpr int kStoreThreads = 256;
constexpr int kStoreRows = 4;

template <typename Vec>
__global__ void __launch_bounds__(kStoreThreads) cache_store_kernel(const dspark_cache_store_args a, int es) {
    const int vpe = (int)sizeof(Vec) / es;  // elements of a piece
    const int per_head = a.D / vpe, per_row = a.H * per_head;
    const int row0 = blockIdx.x * kStoreRows;
    const int rows = min(kStoreRows, a.N - row0);
    const long long limit = (long long)a.n_pages * a.page;
    for (int idx = threadIdx.x; idx < rows * 2 * per_row; idx += kStoreThreads) {
        const int row = row0 + idx / (2 * per_row);
        int rest = idx % (2 * per_row);
        const bool is_v = rest >= per_row;
        if (is_v) rest -= per_row;
        const int h = rest / per_head, e = (rest % per_head) * vpe;
        const int slot = a.slot[row];
        if (slot < 0) continue;
        if (slot >= limit) {
            set_err(a.err, DSPARK_ERR_RANGE);
            continue;
        }
        const long long from = is_v ? row * a.v_row + h * a.v_head + e : row * a.k_row + h * a.k_head + e;
        const int pg = slot / a.page, off = slot % a.page;
        const long long to = (((long long)pg * a.H + h) * a.page + off) * a.D + e;
        const char *src = static_cast<const char *>(is_v ? a.v : a.k) + from * es;
        char *dst = static_cast<char *>(is_v ? a.v_cache : a.k_cache) + to * es;
        *reinterpret_cast<Vec *>(dst) = __ldcs(reinterpret_cast<const Vec *>(src));
    }
}

}  // namespace

cudaError_t launch_page_map(const dspark_page_map_args &a, cudaStream_t s) {
    const size_t smem = sizeof(int) * 3 * (size_t)(a.R + 1);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(page_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const int items = a.N > a.R + 1 ? a.N : a.R + 1;
    int blocks = (items + kMapThreads - 1) / kMapThreads;
    if (blocks > sm_count()) blocks = sm_count();
    page_map_kernel<<<blocks, kMapThreads, smem, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_store(const dspark_cache_store_args &a, cudaStream_t s) {
    const int es = a.dtype == DSPARK_BF16 ? 2 : 4;
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                          reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache) |
                          (uintptr_t)((a.k_row | a.k_head | a.v_row | a.v_head | a.D) * es);
    const int blocks = (a.N + kStoreRows - 1) / kStoreRows;
    if ((all & 15) == 0) cache_store_kernel<uint4><<<blocks, kStoreThreads, 0, s>>>(a, es);
    else if (es == 4) cache_store_kernel<unsigned int><<<blocks, kStoreThreads, 0, s>>>(a, es);
    else cache_store_kernel<unsigned short><<<blocks, kStoreThreads, 0, s>>>(a, es);
    return cudaGetLastError();
}

}  // namespace dspark
