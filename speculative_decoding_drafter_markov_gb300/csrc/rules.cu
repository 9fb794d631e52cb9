// rules.cu -- repetition penalties, biases and grammar masks on the target's
// logits, between the target's pass and the verification.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace dspark {

namespace {

// One CTA takes one request, one slice of the vocabulary and a run of the
// request's rows.  It counts the request's text once, into a word per entry of
// its slice in shared memory, and then passes over the slice of each row: the
// counts are shared by the rows, and what a row continues is added before its
// pass (and what only the row before continued taken out: a chain only adds).
// Beside the logits' one read and one write there is the text, read once per
// slice from L2; a 16-byte piece whose entries are all forbidden is not read.
// Bound by HBM at the large end.
constexpr int kRulesThreads = 256;
constexpr int kBiasList = 256;  // bias entries of a slice kept in shared memory
constexpr uint32_t kPromptBit = 1u << 31, kBiasBit = 1u << 30, kCountMask = kBiasBit - 1;

struct Bias {
    const int *id;      // the slice's entries in shared memory, in their order,
    const float *val;
    int n;              // or, when they are more than fit there, all of the
};                      // request's entries in global memory

struct RowRules {
    float rep, inv_rep, freq, pres;
};

__device__ __noinline__ float biased(float z, int v, Bias b) {
    for (int i = 0; i < b.n; ++i)
        if (b.id[i] == v) z += b.val[i];
    return z;
}

__device__ __forceinline__ float apply(float z, uint32_t word, int v, const RowRules &k, const Bias &b) {
    const uint32_t c = word & kCountMask;
    if (word & (kPromptBit | kCountMask)) z *= z > 0.f ? k.inv_rep : k.rep;
    z = fmaf(-k.freq, (float)c, z);
    if (c) z -= k.pres;
    if (word & kBiasBit) z = biased(z, v, b);
    return z;
}

// 16 bytes of logits
template <typename T>
struct Piece;
template <>
struct Piece<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void get(const uint4 &v, float (&z)[N]) {
        z[0] = __uint_as_float(v.x), z[1] = __uint_as_float(v.y), z[2] = __uint_as_float(v.z), z[3] = __uint_as_float(v.w);
    }
    __device__ static __forceinline__ uint4 put(const float (&z)[N]) {
        return make_uint4(__float_as_uint(z[0]), __float_as_uint(z[1]), __float_as_uint(z[2]), __float_as_uint(z[3]));
    }
};
template <>
struct Piece<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void get(const uint4 &v, float (&z)[N]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) z[2 * i] = __uint_as_float(w[i] << 16), z[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    __device__ static __forceinline__ uint4 put(const float (&z)[N]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(z[2 * i], z[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&two);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ void put(float *p, float z) { *p = z; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float z) { *p = __float2bfloat16_rn(z); }

// kVec: rows of T and out start on 16-byte boundaries
template <typename T, bool kVec>
__global__ void __launch_bounds__(kRulesThreads) logit_rules_kernel(const dspark_logit_rules_args a, int slice) {
    extern __shared__ __align__(16) uint32_t word[];  // [slice]
    __shared__ int bias_id[kBiasList];
    __shared__ float bias_val[kBiasList];
    __shared__ int bias_n;
    const int tid = threadIdx.x, lane = tid & 31;
    const int r = blockIdx.y, v0 = blockIdx.x * slice, v1 = min(a.V, v0 + slice);
    // the request's numbers, all loads in flight together
    const int row0 = a.row_start[r], row_end = a.row_start[r + 1];
    RowRules k;
    k.rep = a.rep ? a.rep[r] : 1.f;
    k.freq = a.freq ? a.freq[r] : 0.f;
    k.pres = a.pres ? a.pres[r] : 0.f;
    int n = a.hist ? a.hist_len[r] : 0, np = a.hist && a.prompt_len ? a.prompt_len[r] : 0;
    int b0 = a.bias_start ? a.bias_start[r] : 0, b1 = a.bias_start ? a.bias_start[r + 1] : 0;
    if (row0 == row_end) return;
    const bool report = tid == 0 && blockIdx.x == 0 && blockIdx.z == 0;
    if (row0 < 0 || row_end < row0 || row_end > a.N || (a.mask && row_end - row0 > 64 * a.W)) {
        if (report) set_err(a.err, DSPARK_ERR_RANGE);
        return;
    }
    const int rows = row_end - row0;
    const int j0 = (int)((long long)rows * blockIdx.z / gridDim.z), j1 = (int)((long long)rows * (blockIdx.z + 1) / gridDim.z);
    if (n < 0 || n > a.max_hist || np < 0 || np > n) {
        if (report) set_err(a.err, DSPARK_ERR_RANGE);
        n = max(0, min(n, a.max_hist));
        np = max(0, min(np, n));
    }
    if (b0 < 0 || b1 < b0 || b1 > a.n_bias) {
        if (report) set_err(a.err, DSPARK_ERR_RANGE);
        b0 = b1 = 0;
    }
    if (j0 == j1) return;
    k.inv_rep = 1.f / k.rep;
    const bool penal = k.rep != 1.f || k.freq != 0.f || k.pres != 0.f;
    const bool counted = penal || b1 > b0;  // the entries' words are in use
    Bias bias{bias_id, bias_val, 0};

    if (counted) {
        for (int i = 4 * tid; i < slice; i += 4 * kRulesThreads) *reinterpret_cast<uint4 *>(word + i) = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        if (penal) {
            const int32_t *text = a.hist + (size_t)r * a.max_hist;
#pragma unroll 8
            for (int i = tid; i < n; i += kRulesThreads) {
                const int v = text[i];
                if (v < 0 || v >= a.V) set_err(a.err, DSPARK_ERR_RANGE);
                if (v >= v0 && v < v1) {
                    if (i < np) atomicOr(&word[v - v0], kPromptBit);
                    else atomicAdd(&word[v - v0], 1u);
                }
            }
        }
        if (b1 > b0 && tid < 32) {  // one warp, so that the list keeps the entries' order
            int found = 0;
            for (int i = b0; i < b1; i += 32) {
                const int v = i + lane < b1 ? a.bias_id[i + lane] : v0;
                if (v < 0 || v >= a.V) set_err(a.err, DSPARK_ERR_RANGE);
                const bool in = i + lane < b1 && v >= v0 && v < v1;
                const unsigned who = __ballot_sync(0xffffffffu, in);
                const int at = found + __popc(who & ((1u << lane) - 1));
                if (in) {
                    atomicOr(&word[v - v0], kBiasBit);
                    if (at < kBiasList) {
                        bias_id[at] = v;
                        bias_val[at] = a.bias_val[i + lane];
                    }
                }
                found += __popc(who);
            }
            if (lane == 0) bias_n = found;
        } else if (tid == 0) {
            bias_n = 0;
        }
        __syncthreads();
        bias.n = bias_n;
        if (bias.n > kBiasList) bias = Bias{a.bias_id + b0, a.bias_val + b0, b1 - b0};
    }

    const int words = (a.V + 31) / 32;
    const bool path = penal && a.tok;
    auto add = [&](int at, uint32_t by) {  // drafted row `at` joins or leaves the path
        const int v = a.tok[row0 + at];
        if (v < 0 || v >= a.V) set_err(a.err, DSPARK_ERR_RANGE);
        if (v >= v0 && v < v1) atomicAdd(&word[v - v0], by);
    };
    for (int j = j0; j < j1; ++j) {
        const int row = row0 + j;
        if (path && !a.mask) {
            // rows 1 .. j; those before j are in already, but for the run's first row
            for (int at = j == j0 ? 1 : j; at <= j; ++at) {
                if (at == 0) continue;
                const int v = a.tok[row0 + at];
                if (v >= v0 && v < v1) {  // the same for all threads: few rows touch a slice
                    __syncthreads();
                    if (tid == 0) add(at, 1u);
                    __syncthreads();
                } else if (tid == 0 && (v < 0 || v >= a.V)) {
                    set_err(a.err, DSPARK_ERR_RANGE);
                }
            }
        } else if (path) {
            const uint64_t *now = a.mask + (size_t)row * a.W, *was = now - a.W;
            for (int at = tid; at < (rows + kRulesThreads - 1) / kRulesThreads * kRulesThreads; at += kRulesThreads) {
                int change = 0;
                if (at > 0 && at < rows) {
                    change = (int)((now[at >> 6] >> (at & 63)) & 1);
                    if (j > j0) change -= (int)((was[at >> 6] >> (at & 63)) & 1);
                }
                __syncthreads();  // the row before is done
                if (change) add(at, (uint32_t)change);
            }
            __syncthreads();
        }
        const uint32_t *allow = nullptr;
        if (a.allow) {
            const int m = a.allow_row[row];
            if (m >= a.n_allow) {
                if (tid == 0) set_err(a.err, DSPARK_ERR_RANGE);
            } else if (m >= 0) {
                allow = a.allow + (size_t)m * words;
            }
        }
        const T *src = static_cast<const T *>(a.T) + (size_t)row * a.V;
        T *dst = static_cast<T *>(a.out) + (size_t)row * a.V;
        if (kVec) {
            constexpr int E = Piece<T>::N, U = 4;
            constexpr uint32_t kAll = (1u << E) - 1;
            for (int vb = v0 + E * tid; vb < v1; vb += U * E * kRulesThreads) {
                uint32_t ok[U];
                uint4 raw[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = vb + u * E * kRulesThreads;
                    ok[u] = v < v1 ? kAll : 0u;
                    if (allow && v < v1) ok[u] = (allow[v >> 5] >> (v & 31)) & kAll;
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = vb + u * E * kRulesThreads;
                    raw[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (ok[u]) raw[u] = __ldcs(reinterpret_cast<const uint4 *>(src + v));
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = vb + u * E * kRulesThreads;
                    if (v >= v1) break;
                    uint4 res = raw[u];
                    uint32_t w[E], any = 0;
                    if (counted) {
#pragma unroll
                        for (int i = 0; i < E; i += 4) {
                            const uint4 q = *reinterpret_cast<const uint4 *>(word + (v - v0) + i);
                            w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
                            any |= q.x | q.y | q.z | q.w;
                        }
                    }
                    if (any || ok[u] != kAll) {
                        float z[E];
                        Piece<T>::get(res, z);
                        if (any) {
#pragma unroll
                            for (int i = 0; i < E; ++i)
                                if (w[i]) z[i] = apply(z[i], w[i], v + i, k, bias);
                        }
#pragma unroll
                        for (int i = 0; i < E; ++i)
                            if (!((ok[u] >> i) & 1)) z[i] = -INFINITY;
                        res = Piece<T>::put(z);
                    }
                    __stcs(reinterpret_cast<uint4 *>(dst + v), res);
                }
            }
        } else {
            constexpr int U = 8;
            for (int vb = v0 + tid; vb < v1; vb += U * kRulesThreads) {
                float z[U];
                bool ok[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = vb + u * kRulesThreads;
                    z[u] = v < v1 ? to_f32(src[v]) : 0.f;
                    ok[u] = !allow || v >= v1 || ((allow[v >> 5] >> (v & 31)) & 1);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int v = vb + u * kRulesThreads;
                    if (v >= v1) break;
                    if (counted) {
                        const uint32_t w = word[v - v0];
                        if (w) z[u] = apply(z[u], w, v, k, bias);
                    }
                    put(dst + v, ok[u] ? z[u] : -INFINITY);
                }
            }
        }
    }
}

template <typename T>
cudaError_t launch_as(const dspark_logit_rules_args &a, cudaStream_t s) {
    // Slices as large as leave every SM three CTAs (a slice's words take 4 bytes
    // an entry, and the text is read once per slice); where requests are few the
    // rows are spread too, at the price of counting the text for each run.
    const long long want = 3ll * sm_count();
    int slice = 8192;
    while (slice > 1024 && (long long)a.R * ((a.V + slice - 1) / slice) < want) slice /= 2;
    const int slices = (a.V + slice - 1) / slice;
    const long long per = (a.N + a.R - 1) / a.R;
    long long runs = want / ((long long)slices * a.R);
    if (runs > per) runs = per;
    if (runs < 1) runs = 1;
    const dim3 grid(slices, a.R, (unsigned)runs);
    const size_t smem = sizeof(uint32_t) * slice;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.T) | reinterpret_cast<uintptr_t>(a.out) | ((uintptr_t)a.V * sizeof(T));
    if ((at & 15) == 0) logit_rules_kernel<T, true><<<grid, kRulesThreads, smem, s>>>(a, slice);
    else logit_rules_kernel<T, false><<<grid, kRulesThreads, smem, s>>>(a, slice);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logit_rules(const dspark_logit_rules_args &a, cudaStream_t s) {
    return a.dtype == DSPARK_BF16 ? launch_as<__nv_bfloat16>(a, s) : launch_as<float>(a, s);
}

}  // namespace dspark
