// rules.cu -- repetition penalties, biases and grammar masks on the target's
// logits, between the target's pass and the verification.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"

namespace dspark {

namespace {

// One CTA takes one request and one slice of the vocabulary.  It counts the
// request's text once, into a word per entry of its slice in shared memory, and
// then passes over the slice of each of the request's rows: the counts are
// shared by the rows, and a row's own drafted tokens are added before its pass
// and taken out after it (a chain only ever adds).  Work beside the logits'
// one read and one write: the text, read once per slice from L2.
constexpr int kRulesThreads = 256;
constexpr int kBiasList = 256;  // bias entries of a slice kept in shared memory
constexpr uint32_t kPromptBit = 1u << 31, kBiasBit = 1u << 30, kCountMask = kBiasBit - 1;

__device__ __forceinline__ void put(float *p, float z) { *p = z; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float z) { *p = __float2bfloat16_rn(z); }

struct Bias {
    const int *id;      // the slice's entries in shared memory, in their order,
    const float *val;
    int n;              // or, when they are more than fit there, all of the
};                      // request's entries in global memory

struct RowRules {
    float rep, freq, pres;
    bool counted;  // any penalty, or a bias: the entries' words are in use
};

__device__ __forceinline__ float apply(float z, uint32_t word, int v, const RowRules &k, const Bias &b) {
    if (word == 0) return z;
    const uint32_t c = word & kCountMask;
    if (word & (kPromptBit | kCountMask)) z = z > 0.f ? z / k.rep : z * k.rep;
    z -= k.freq * (float)c;
    if (c) z -= k.pres;
    if (word & kBiasBit)
        for (int i = 0; i < b.n; ++i)
            if (b.id[i] == v) z += b.val[i];
    return z;
}

template <typename T>
__global__ void __launch_bounds__(kRulesThreads) logit_rules_kernel(const dspark_logit_rules_args a, int slice, bool vec) {
    extern __shared__ __align__(16) uint32_t word[];  // [slice]
    __shared__ int bias_id[kBiasList];
    __shared__ float bias_val[kBiasList];
    __shared__ int bias_n;
    const int tid = threadIdx.x, lane = tid & 31;
    const int r = blockIdx.y, v0 = blockIdx.x * slice, v1 = min(a.V, v0 + slice);
    const int row0 = a.row_start[r], row1 = a.row_start[r + 1];
    if (row0 == row1) return;
    if (row0 < 0 || row1 < row0 || row1 > a.N || (a.mask && row1 - row0 > 64 * a.W)) {
        if (tid == 0) set_err(a.err, DSPARK_ERR_RANGE);
        return;
    }
    RowRules k;
    k.rep = a.rep ? a.rep[r] : 1.f;
    k.freq = a.freq ? a.freq[r] : 0.f;
    k.pres = a.pres ? a.pres[r] : 0.f;
    const bool penal = k.rep != 1.f || k.freq != 0.f || k.pres != 0.f;
    int b0 = 0, b1 = 0;
    if (a.bias_start) {
        b0 = a.bias_start[r];
        b1 = a.bias_start[r + 1];
        if (b0 < 0 || b1 < b0 || b1 > a.n_bias) {
            if (tid == 0) set_err(a.err, DSPARK_ERR_RANGE);
            b0 = b1 = 0;
        }
    }
    int n = 0, np = 0;  // the text, and its prompt part
    if (a.hist) {
        n = a.hist_len[r];
        np = a.prompt_len ? a.prompt_len[r] : 0;
        if (n < 0 || n > a.max_hist || np < 0 || np > n) {
            if (tid == 0) set_err(a.err, DSPARK_ERR_RANGE);
            n = max(0, min(n, a.max_hist));
            np = max(0, min(np, n));
        }
    }
    k.counted = penal || b1 > b0;
    Bias bias{bias_id, bias_val, 0};

    if (k.counted) {
        for (int i = tid; i < slice; i += kRulesThreads) word[i] = 0;
        __syncthreads();
        if (penal && a.hist) {
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
    for (int row = row0; row < row1; ++row) {
        const int j = row - row0;
        if (path && j > 0) {
            // what this row continues, less what the row before did
            __syncthreads();
            auto change = [&](int at, int by) {
                const int v = a.tok[row0 + at];
                if (v < 0 || v >= a.V) set_err(a.err, DSPARK_ERR_RANGE);
                if (v >= v0 && v < v1) atomicAdd(&word[v - v0], (uint32_t)by);
            };
            if (!a.mask) {
                if (tid == 0) change(j, 1);
            } else {
                for (int at = tid; at < row1 - row0; at += kRulesThreads) {
                    if (at == 0) continue;
                    const uint64_t *now = a.mask + (size_t)row * a.W, *was = now - a.W;
                    const int n = (int)((now[at >> 6] >> (at & 63)) & 1);
                    const int w = (int)((was[at >> 6] >> (at & 63)) & 1);
                    if (n != w) change(at, n - w);
                }
            }
            __syncthreads();
        } else if (path && a.mask) {  // the first row continues nothing but what its mask says
            for (int at = tid; at < row1 - row0; at += kRulesThreads)
                if (at > 0 && ((a.mask[(size_t)row * a.W + (at >> 6)] >> (at & 63)) & 1)) {
                    const int v = a.tok[row0 + at];
                    if (v < 0 || v >= a.V) set_err(a.err, DSPARK_ERR_RANGE);
                    if (v >= v0 && v < v1) atomicAdd(&word[v - v0], 1u);
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
#pragma unroll 4
        for (int v = v0 + tid; v < v1; v += kRulesThreads) {
            float z = to_f32(src[v]);
            if (k.counted) z = apply(z, word[v - v0], v, k, bias);
            if (allow && !((allow[v >> 5] >> (v & 31)) & 1)) z = -INFINITY;
            put(dst + v, z);
        }
    }
}

}  // namespace

cudaError_t launch_logit_rules(const dspark_logit_rules_args &a, cudaStream_t s) {
    const int slice = 8192;
    const bool vec = false;
    const dim3 grid((a.V + slice - 1) / slice, a.R);
    const size_t smem = sizeof(uint32_t) * slice;
    if (a.dtype == DSPARK_BF16) logit_rules_kernel<__nv_bfloat16><<<grid, kRulesThreads, smem, s>>>(a, slice, vec);
    else logit_rules_kernel<float><<<grid, kRulesThreads, smem, s>>>(a, slice, vec);
    return cudaGetLastError();
}

}  // namespace dspark
