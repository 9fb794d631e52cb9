// paged.cu -- the paged key-value cache around the target's pass: the batch map
// of a cycle (pages, row starts, slots, positions, ancestor masks) and the
// write of the rows' keys and values.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "paged.cuh"
#include "target.h"

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
// Bound by latency, a chain of loads, a scan and a store: 4 requests 3.0 us, 96 prompts
// of up to 32768 rows 5.5, 512 trees of up to 64 rows 8.2, of which 3 are the walk from
// a row to its root (the parents staged in shared memory first gained nothing).  With
// 256 threads 8192 requests take 25 us; 128, 512 and 1024 were no faster.
constexpr int kMapThreads = 256;

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

// pages of a request; the sum of two non-negative 32-bit sizes fits 32 bits unsigned
__device__ __forceinline__ unsigned need_of(const dspark_page_map_args &a, const Page &page, int r) {
    const unsigned t = (unsigned)a.len[r] + (unsigned)a.rows[r], q = page.of(t);
    return q + (t != q * page.size);
}

__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const dspark_page_map_args a, const Page page) {
    extern __shared__ int sh[];
    after_predecessor();
    const int R = a.R;
    const MapSums s{sh, sh + (R + 1), sh + 2 * (R + 1)};
    __shared__ unsigned wsum[2][3][kMapThreads / 32];
    __shared__ int bad_any;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) bad_any = 0;
    const int before = *a.n_free;

    // running sums, a request per thread at a time; sums beyond 2^31 - 1, of which no
    // call is good, stay there
    auto add = [](unsigned x, unsigned y) { return min(x + y, 0x7fffffffu); };
    unsigned total[3] = {0, 0, 0};
    bool bad = false;
    __syncthreads();
    for (int r0 = 0, turn = 0; r0 < R; r0 += kMapThreads, turn ^= 1) {
        const int r = r0 + tid;
        unsigned v[3] = {0, 0, 0};
        if (r < R) {
            const int len = a.len[r], rows = a.rows[r], held = a.held[r];
            const unsigned need = need_of(a, page, r);
            if (len < 0 || rows < 0 || held < 0 || held > a.max_pages || need > (unsigned)a.max_pages || (a.mask && rows > 64 * a.W)) {
                bad = true;
            } else {
                v[0] = rows;
                v[1] = max(0, held - (int)need);
                v[2] = max(0, (int)need - held);
            }
        }
        unsigned inc[3] = {v[0], v[1], v[2]};
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const unsigned y = __shfl_up_sync(0xffffffffu, inc[i], d);
                if (lane >= d) inc[i] = add(inc[i], y);
            }
        if (lane == 31)
#pragma unroll
            for (int i = 0; i < 3; ++i) wsum[turn][i][warp] = inc[i];
        __syncthreads();
        unsigned base[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            unsigned b = total[i];
#pragma unroll
            for (int w = 0; w < kMapThreads / 32; ++w) {
                const unsigned x = wsum[turn][i][w];
                if (w < warp) b = add(b, x);
                total[i] = add(total[i], x);
            }
            base[i] = b + inc[i] - v[i];
        }
        if (r < R) {
            s.rows[r] = (int)base[0];
            s.less[r] = (int)base[1];
            s.more[r] = (int)base[2];
        }
    }
    if (bad) bad_any = 1;
    if (tid == 0) {
        s.rows[R] = (int)total[0];
        s.less[R] = (int)total[1];
        s.more[R] = (int)total[2];
    }
    __syncthreads();

    const bool fail = bad_any || total[0] > (unsigned)a.N || (a.parents && total[0] > (unsigned)a.n_parents) || before < 0 ||
                      (unsigned)before + total[1] > (unsigned)a.n_pages || total[2] > (unsigned)before + total[1];
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
        return a.table[(size_t)r * a.max_pages + need_of(a, page, r) + (k - s.less[r])];
    };
    auto page_of = [&](int k) {  // the k-th page taken
        return k < m ? given(k) : a.free_list[before - 1 - (k - m)];
    };
    // whoever moves a page, or stores into it, reports one that the cache has not
    auto is_page = [&](int pg) {
        const bool ok = (unsigned)pg < (unsigned)a.n_pages;
        if (!ok) set_err(a.err, DSPARK_ERR_RANGE);
        return ok;
    };

    if (first == 0) *a.n_free_out = after - taken;
    for (int r = first; r <= R; r += step) {
        a.row_start[r] = s.rows[r];
        if (r < R) a.held_out[r] = (int)need_of(a, page, r);
    }
    for (int k = first; k < m; k += step) {
        const int pg = given(k);
        is_page(pg);
        a.free_list[after - 1 - k] = pg;
    }
    for (int k = first; k < taken; k += step) {
        const int r = holder(s.more, R, k), pg = page_of(k);
        is_page(pg);
        a.table[(size_t)r * a.max_pages + a.held[r] + (k - s.more[r])] = pg;
    }
    for (int i = first; i < a.N; i += step) {
        int slot = -1, pos = 0;
        if (i < s.rows[R]) {
            const int r = holder(s.rows, R, i), start = s.rows[r], j = i - start;
            const int t = a.len[r] + j, pi = (int)page.of(t), held = a.held[r];
            const int pg = pi < held ? a.table[(size_t)r * a.max_pages + pi] : page_of(s.more[r] + pi - held);
            if (is_page(pg)) slot = pg * a.page + (t - pi * a.page);
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
// A copy of 2 N H D elements: bound by HBM (read once, written once).  A thread has
// one 16-byte piece of a row -- keys or values, head and columns are found once --
// and takes it from kRows rows, all reads under way together; neighbouring threads
// have neighbouring pieces.  24 prompts of up to 8192 rows, 8 heads of 128, bf16: 24.3 us,
// 5.7 TB/s (one row a thread: 31.5 us); 64 requests of up to 9 rows: 2.1 us.
constexpr int kStoreThreads = 256;

template <typename Vec, int kRows>
__global__ void __launch_bounds__(kStoreThreads) cache_store_kernel(const dspark_cache_store_args a, const Page page, int es) {
    after_predecessor();
    const int vpe = (int)sizeof(Vec) / es;  // elements of a piece
    const int per_head = a.D / vpe, per_row = a.H * per_head;
    int piece = blockIdx.y * kStoreThreads + threadIdx.x;
    if (piece >= 2 * per_row) return;
    const bool values = piece >= per_row;
    if (values) piece -= per_row;
    const int h = piece / per_head, e = (piece - h * per_head) * vpe;
    const char *src = static_cast<const char *>(values ? a.v : a.k) + (h * (values ? a.v_head : a.k_head) + e) * es;
    char *dst = static_cast<char *>(values ? a.v_cache : a.k_cache) + e * es;
    const long long row_bytes = (values ? a.v_row : a.k_row) * es;
    const unsigned limit = (unsigned)min((long long)a.n_pages * a.page, 0x80000000ll);
    const int row0 = blockIdx.x * kRows;
    int slot[kRows];
    Vec v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) slot[i] = row0 + i < a.N ? a.slot[row0 + i] : -1;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (slot[i] >= 0 && (unsigned)slot[i] >= limit) {
            set_err(a.err, DSPARK_ERR_RANGE);
            slot[i] = -1;
        }
        if (slot[i] >= 0) v[i] = __ldcs(reinterpret_cast<const Vec *>(src + (row0 + i) * row_bytes));
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (slot[i] < 0) continue;
        const int pg = (int)page.of(slot[i]), off = slot[i] - pg * a.page;
        *reinterpret_cast<Vec *>(dst + (((long long)pg * a.H + h) * a.page + off) * a.D * es) = v[i];
    }
}

template <typename Vec>
cudaError_t store_as(const dspark_cache_store_args &a, const Page &page, int es, cudaStream_t s) {
    const int pieces = 2 * a.H * (a.D / ((int)sizeof(Vec) / es)), y = (pieces + kStoreThreads - 1) / kStoreThreads;
    // eight rows a thread where that leaves every SM a few CTAs, else one
    const bool many = (long long)a.N * y >= 8ll * 4 * sm_count();
    return many ? launch_close(cache_store_kernel<Vec, 8>, dim3((a.N + 7) / 8, y), kStoreThreads, 0, s, a, page, es)
                : launch_close(cache_store_kernel<Vec, 1>, dim3(a.N, y), kStoreThreads, 0, s, a, page, es);
}

}  // namespace

cudaError_t launch_page_map(const dspark_page_map_args &a, cudaStream_t s) {
    const size_t smem = sizeof(int) * 3 * (size_t)(a.R + 1);
    if (smem > 32 * 1024) {  // well below the 48 KB, which the kernel's own variables share
        cudaError_t e = cudaFuncSetAttribute(page_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const int items = a.N > a.R + 1 ? a.N : a.R + 1;
    int blocks = (items + kMapThreads - 1) / kMapThreads;
    if (blocks > 4 * sm_count()) blocks = 4 * sm_count();
    return launch_close(page_map_kernel, blocks, kMapThreads, smem, s, a, page_of_size(a.page));
}

cudaError_t launch_cache_store(const dspark_cache_store_args &a, cudaStream_t s) {
    const int es = a.dtype == DSPARK_BF16 ? 2 : 4;
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                          reinterpret_cast<uintptr_t>(a.k_cache) | reinterpret_cast<uintptr_t>(a.v_cache) |
                          (uintptr_t)((a.k_row | a.k_head | a.v_row | a.v_head | a.D) * es);
    const Page page = page_of_size(a.page);
    if ((all & 15) == 0) return store_as<uint4>(a, page, es, s);
    return es == 4 ? store_as<unsigned int>(a, page, es, s) : store_as<unsigned short>(a, page, es, s);
}

}  // namespace dspark
