// cache4.cu -- the write of the rows' keys and values into a cache of 4 bits.
//
// One read of the rows and a write of 9/32 of it; beside that a maximum over 16 elements, the
// nearest scale, and per element an exact rounding, two operations in bf16.  24 prompts of
// up to 8192 rows (8 heads of 128, keys and values, 159 MB moved) take 29 us, 5.5 TB/s, 0.81 of a plain copy's
// rate, with 70 % of the issue slots used, most stalls for the rows (5.1 of 12 cycles an instruction).  That is with the values that the
// cache then holds written back; by events around a call (4 us more) 33 us with them and 23 without (89 MB: instructions bound that
// call), in fp32 58 and 46.  A cycle's rows (64 requests of up to 9) take 4.7 us, which is the call on the host.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "cache4.cuh"
#include "common.cuh"
#include "paged.cuh"
#include "target.h"

namespace dspark {

namespace {

// A thread has the 16 elements of a row that share a scale -- keys or values, head and columns
// are found once -- and takes them from kRows rows, all reads under way together.  (8 elements a
// thread, its neighbour with the other 8, four rows: 30.9 us for the prompts above; 16 and four rows 30.0,
// two rows 29.0.  With the row's number compared as a difference in place of an unsigned sum 41 against 33 us at
// that stage: the four slots were then read one by one.)
constexpr int kThreads = 128;

template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void load_each(const __nv_bfloat16 *p) {
        const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
        v.x = u[0] | (unsigned)u[1] << 16, v.y = u[2] | (unsigned)u[3] << 16;
        v.z = u[4] | (unsigned)u[5] << 16, v.w = u[6] | (unsigned)u[7] << 16;
    }
    // bits of the largest magnitude as a float; infinities and NaN are the largest of all
    __device__ __forceinline__ unsigned most() const {
        const unsigned m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
        return max(m << 16, m & 0xffff0000u);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    // n s is a bf16 number: its high half is all of it
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&x)[8]) {
        unsigned w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632);
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float coded(float x, float, float inv) { return cache4::coded_bf16(x, inv); }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldcs(reinterpret_cast<const float4 *>(p));
        b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void load_each(const float *p) {
        a = make_float4(p[0], p[1], p[2], p[3]);
        b = make_float4(p[4], p[5], p[6], p[7]);
    }
    __device__ __forceinline__ unsigned most() const {
        float x[8];
        get(x);
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[8]) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
    static __device__ __forceinline__ float coded(float x, float s, float inv) { return 12582920.f + cache4::whole_of(x, s, inv); }
};

template <typename T, bool kWide, int kRows>
__global__ void __launch_bounds__(kThreads) cache_store4_kernel(const dspark_cache_store4_args a, const Page page) {
    after_predecessor();
    const int per_head = a.D / 16, per_row = a.H * per_head;
    int piece = blockIdx.y * kThreads + threadIdx.x;
    const bool in = piece < 2 * per_row;
    const bool values = piece >= per_row;
    if (values) piece -= per_row;
    const int h = piece / per_head, e = (piece - h * per_head) * 16;
    const T *src = static_cast<const T *>(values ? a.v : a.k) + (values ? a.v_head : a.k_head) * h + e;
    const long long row = values ? a.v_row : a.k_row;
    // this thread's codes and scale of the first token of page 0; what a page and a token add
    const long long page_bytes = cache4::page_bytes(a.page, a.D), page_step = page_bytes * a.H;
    unsigned char *codes = (values ? a.v_cache : a.k_cache) + page_bytes * h + e / 2;
    unsigned char *scales = codes - e / 2 + cache4::code_bytes(a.page, a.D) + e / 16;
    const unsigned code_row = a.D / 2, scale_row = a.D / 16;
    T *held = static_cast<T *>(values ? a.v_out : a.k_out);
    const unsigned slots = slots_of(a.n_pages, a.page);
    const int row0 = blockIdx.x * kRows;
    int slot[kRows];
    Eight<T> v[kRows][2];
#pragma unroll
    for (int i = 0; i < kRows; ++i) slot[i] = in && (unsigned)row0 + i < (unsigned)a.N ? a.slot[row0 + i] : -1;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        slot[i] = checked_slot(slot[i], slots, a.err);
        if (slot[i] < 0) continue;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (kWide) v[i][p].load(src + (row0 + i) * row + 8 * p);
            else v[i][p].load_each(src + (row0 + i) * row + 8 * p);
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        if (slot[i] < 0) continue;
        const unsigned most = max(v[i][0].most(), v[i][1].most());
        const bool beyond = __uint_as_float(most) > cache4::kMostHeld;  // the largest scale
        const unsigned byte = cache4::scale_byte(__uint_as_float(most));
        const float s = cache4::scale_of(byte), inv = __fdividef(1.f, s);  // (a last bit or two is nothing to what takes it)
        const unsigned pg = page.of(slot[i]), off = slot[i] - pg * page.size;
        const long long at = pg * page_step;
        unsigned word[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float x[8];
            v[i][p].get(x);
            if (beyond) {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = fminf(fmaxf(x[k], -cache4::kMostHeld), cache4::kMostHeld);
            }
            unsigned code[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) code[k] = __float_as_uint(Eight<T>::coded(x[k], s, inv));
            // elements 0 4 1 5 in the low halves of the four bytes, 2 6 3 7 in the high ones
            const unsigned low = __byte_perm(__byte_perm(code[0], code[4], 0x0040), __byte_perm(code[1], code[5], 0x0040), 0x5410);
            const unsigned high = __byte_perm(__byte_perm(code[2], code[6], 0x0040), __byte_perm(code[3], code[7], 0x0040), 0x5410);
            word[p] = byte == cache4::kNoNumbers ? 0x88888888u : low + 16u * high;
            if (held) {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = byte == cache4::kNoNumbers ? s : (__uint_as_float(code[k]) - 12582920.f) * s;
                Eight<T>::store(held + (row0 + i) * ((long long)a.H * a.D) + h * a.D + e + 8 * p, x);
            }
        }
        *reinterpret_cast<uint2 *>(codes + at + (unsigned long long)off * code_row) = make_uint2(word[0], word[1]);
        scales[at + (unsigned long long)off * scale_row] = (unsigned char)byte;
    }
}

template <typename T, bool kWide>
cudaError_t store_as(const dspark_cache_store4_args &a, const Page &page, cudaStream_t s) {
    const int pieces = 2 * a.H * (a.D / 16), y = (pieces + kThreads - 1) / kThreads;
    // two rows a thread where that leaves every SM a few CTAs, else one
    const bool many = (long long)a.N * y >= 2ll * 8 * sm_count();
    return many ? launch_close(cache_store4_kernel<T, kWide, 2>, dim3((a.N - 1) / 2 + 1, y), kThreads, 0, s, a, page)
                : launch_close(cache_store4_kernel<T, kWide, 1>, dim3(a.N, y), kThreads, 0, s, a, page);
}

}  // namespace

cudaError_t launch_cache_store4(const dspark_cache_store4_args &a, cudaStream_t s) {
    const int es = a.dtype == DSPARK_BF16 ? 2 : 4;
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                          (uintptr_t)((a.k_row | a.k_head | a.v_row | a.v_head) * es);
    const Page page = page_of_size(a.page);
    const bool wide = (all & 15) == 0;
    if (a.dtype == DSPARK_BF16) return wide ? store_as<__nv_bfloat16, true>(a, page, s) : store_as<__nv_bfloat16, false>(a, page, s);
    return wide ? store_as<float, true>(a, page, s) : store_as<float, false>(a, page, s);
}

}  // namespace dspark
