// rope.cu -- queries, keys and values of the rows on their way into the attention: the
// norm of each head, the rotation by position, the append to the paged cache.
//
// What has to be done is one read and one write of every row; the sines and cosines of a row are
// shared by its heads, so a warp takes a whole row where there are rows enough.  A run of a
// server's cycle (64 requests of up to 9 rows, 32 query heads on 8 of 128) takes 5 us, a launch
// and the trips from slot and position to the store, and 24 prompts of up to 8192 rows (418 MB) 79 us,
// 5.3 TB/s: 0.78 of a plain copy's rate.  There 47 % of the issue slots are used and the DRAM 58 % of
// its cycles; what is left is waiting for the loads of two heads a thread (stalls: 3.8 of 10 cycles an
// instruction for memory, 2.2 for fixed latencies).  Six, seven or eight CTAs an SM by fewer registers took
// 80, 85 and 93 us, warps that stay and fetch the next row's first heads ahead 82 (at 81 us).  Lanes
// beyond a head's pieces carry nothing: with heads of 80 or 96 (8 lanes, 5 or 6 in use) the same rows take
// 79 and 81 us by events around a call, where heads of 128 take 85.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "paged.cuh"
#include "target.h"

namespace dspark {

namespace {

// ---------------------------------------------------------------- angles
// pos freq in turns, modulo one: with F = freq / (2 pi) as a 64-bit binary fraction
// (whole turns dropped) pos F modulo 2^64 is the fraction of a turn, for positions of
// either sign.  F is cut below 2^-64, so the angle is off by pos 2^-64 turns at most.
// The significand of freq (24 bits) times 128 bits of 1 / (2 pi), in words p2 p1 p0.
__device__ __forceinline__ unsigned long long turns_of(float freq) {
    const unsigned long long c1 = 0x28be60db9391054aull, c0 = 0x7f09d5f47d4d3770ull;
    const unsigned bits = __float_as_uint(freq);
    const int e = (bits >> 23) & 255;
    const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
    const unsigned long long p0 = m * c0, low = m * c1, p1 = low + __umul64hi(m, c0);
    const unsigned long long p2 = __umul64hi(m, c1) + (p1 < low);
    const int shift = 214 - (e ? e : 1);  // freq = m 2^(e - 150)
    unsigned long long f = 0;
    if (shift >= 128) f = shift < 192 ? p2 >> (shift - 128) : 0;
    else if (shift > 64) f = (p1 >> (shift - 64)) | (p2 << (128 - shift));
    else if (shift > 0) f = shift == 64 ? p1 : (p0 >> shift) | (p1 << (64 - shift));
    return bits >> 31 ? 0ull - f : f;
}
__device__ __forceinline__ float2 cos_sin(unsigned long long turns, int pos) {
    const long long t = (long long)((unsigned long long)(long long)pos * turns);  // -1/2 .. 1/2 turn
    float s, c;
    sincospif(__ll2float_rn(t) * 0x1p-63f, &s, &c);
    return make_float2(c, s);
}

// ---------------------------------------------------------------- squares beyond fp32
// Where the sum of squares passes fp32 it is formed of (x 2^-96)^2, 2^64 each at most; some |x| is
// 2^60 or more, and only elements below 2^-27 of that lose bits.  1 / root is then between
// 2^-128 and 2^-60, which may be subnormal, so half of 2^-96 goes to x beforehand: x 2^-48 is exact
// wherever the result is a normal number.
constexpr float kDown = 0x1p-96f, kHalfDown = 0x1p-48f;
__device__ __forceinline__ bool beyond_fp32(float sum) { return !(sum <= 3.4e38f); }
// 2^48 / root of the squares' mean and eps: what x 2^-48 is multiplied with
__device__ __forceinline__ float factor_beyond(float scaled, float inv_D, float eps) {
    return rsqrtf(fmaf(scaled, inv_D, eps * kDown * kDown)) * kHalfDown;
}

template <typename T>
__device__ __forceinline__ T round_to(float v);
template <>
__device__ __forceinline__ float round_to(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 round_to(float v) { return __float2bfloat16_rn(v); }

// where a head of a row comes from and goes to
struct Head {
    const void *src;
    void *dst;
    const void *weight;
    bool turn;  // a query or a key
};

// head 0 .. Hq - 1: queries, then H keys, then (with a cache) H values
struct Rows {
    dspark_rope_store_args a;
    Page page;
    int heads;
    unsigned splits;  // parts of a row's heads, each of a warp
    int per_split;    // heads of a part
    template <typename T>
    __device__ __forceinline__ Head head(int h, int i, int slot) const {
        Head x;
        if (h < a.Hq) {
            x.src = static_cast<const T *>(a.q) + i * a.q_row + h * a.q_head;
            x.dst = static_cast<T *>(a.q_out) + i * a.q_out_row + h * a.q_out_head;
            x.weight = a.q_weight;
            x.turn = true;
            return x;
        }
        h -= a.Hq;
        x.turn = h < a.H;
        x.weight = x.turn ? a.k_weight : nullptr;
        if (!x.turn) h -= a.H;
        x.src = x.turn ? static_cast<const T *>(a.k) + i * a.k_row + h * a.k_head : static_cast<const T *>(a.v) + i * a.v_row + h * a.v_head;
        if (a.slot) {
            const int pg = (int)page.of(slot);
            x.dst = static_cast<T *>(x.turn ? a.k_cache : a.v_cache) + (((long long)pg * a.H + h) * a.page + (slot - pg * a.page)) * a.D;
        } else {
            x.dst = static_cast<T *>(a.k_out) + i * a.k_out_row + h * a.k_out_head;
        }
        return x;
    }
};

// ---------------------------------------------------------------- pieces of 16 or 8 bytes
// A warp takes a row's heads, or a part of them, 32 / kLanes heads at a time.  A thread
// has the two pieces of E elements of a head that are rotated together -- E of the first
// half and E of the second, or 2 E neighbours -- so pairs meet in its registers, and a
// norm's sum is formed by the head's kLanes threads.  Sines and cosines are computed once
// per row and part, two pairs a thread, and handed around through shared memory.
constexpr int kWarps = 4, kMaxPairs = DSPARK_ATTN_MAX_D / 2;

template <typename T, int kBytes>
struct PieceOf {
    static constexpr int E = kBytes / (int)sizeof(T);
    unsigned w[kBytes / 4];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kBytes == 16) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
            w[0] = v.x, w[1] = v.y;
        }
    }
    // what other warps read too
    __device__ __forceinline__ void load_shared(const T *p) {
        if constexpr (kBytes == 16) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
            w[0] = v.x, w[1] = v.y;
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (kBytes == 16) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void set(const float2 (&x)[E / 2]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) w[2 * i] = __float_as_uint(x[i].x), w[2 * i + 1] = __float_as_uint(x[i].y);
        } else {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const __nv_bfloat162 two = __floats2bfloat162_rn(x[i].x, x[i].y);
                w[i] = *reinterpret_cast<const unsigned *>(&two);
            }
        }
    }
};

template <typename T, int kBytes, int kLanes, bool kNeighbours>
__global__ void __launch_bounds__(32 * kWarps) rope_store_kernel(const __grid_constant__ Rows r) {
    using P = PieceOf<T, kBytes>;
    constexpr int E = P::E, kHeads = 32 / kLanes;
    __shared__ float2 turned[kWarps][kMaxPairs];
    const dspark_rope_store_args &a = r.a;
    after_predecessor();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = a.rot / 2;
    const long long item = (long long)blockIdx.x * kWarps + warp;
    if (item >= (long long)a.N * r.splits) return;
    const int i = (int)(item / r.splits), part = (int)(item - (long long)i * r.splits);
    // everything that is read at the start is on its way before anything is waited for
    int slot = a.slot ? a.slot[i] : 0;
    const int pos = a.pos[i];
    float freq[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (lane + 32 * k < half) freq[k] = a.freq[lane + 32 * k];
    const int h0 = part * r.per_split, h1 = min(r.heads, h0 + r.per_split);
    // this thread's pieces of a head: pairs j0 .. j0 + E - 1
    const int in_head = lane % kLanes, j0 = in_head * E;
    const bool in = j0 < a.D / 2, turn = j0 < half;
    int at0, at1;
    if (kNeighbours) {
        at0 = 2 * j0;
        at1 = at0 + E;
    } else {
        at0 = turn ? j0 : a.rot + j0 - half;
        at1 = at0 + (turn ? half : (a.D - a.rot) / 2);
    }
    // where the row's queries, keys and values come from and go to
    const T *q_src = static_cast<const T *>(a.q) + i * a.q_row + at0, *k_src = static_cast<const T *>(a.k) + i * a.k_row + at0,
            *v_src = static_cast<const T *>(a.v) + i * a.v_row + at0;
    const int apart = at1 - at0;
    // heads two at a time
    P x[2][2] = {};  // (zeros in the threads beyond D: part of their heads' sums)
    auto fetch = [&](int h, P (&y)[2]) {
        if (h >= h1 || !in) return;
        const T *src = h < a.Hq ? q_src + h * a.q_head : h < a.Hq + a.H ? k_src + (h - a.Hq) * a.k_head : v_src + (h - a.Hq - a.H) * a.v_head;
        y[0].load(src);
        y[1].load(src + apart);
    };
    const int first = h0 + lane / kLanes;
    fetch(first, x[0]);
    fetch(first + kHeads, x[1]);
    if (a.slot) {
        slot = checked_slot(slot, slots_of(a.n_pages, a.page), a.err);
        if (slot < 0) return;
    }
    T *q_dst = static_cast<T *>(a.q_out) + i * a.q_out_row + at0, *k_dst, *v_dst = nullptr;
    long long k_step = a.k_out_head;
    if (a.slot) {
        const int pg = (int)r.page.of(slot);
        const long long at = ((long long)pg * a.H * a.page + (slot - pg * a.page)) * a.D + at0;
        k_dst = static_cast<T *>(a.k_cache) + at;
        v_dst = static_cast<T *>(a.v_cache) + at;
        k_step = (long long)a.page * a.D;
    } else {
        k_dst = static_cast<T *>(a.k_out) + i * a.k_out_row + at0;
    }
    if (h0 < a.Hq + a.H) {
        for (int j = lane, k = 0; j < half; j += 32, ++k)
            turned[warp][j] = cos_sin(turns_of(k == 0 ? freq[0] : k == 1 ? freq[1] : a.freq[j]), pos);
        __syncwarp();
    }
    float c[E], s[E];
#pragma unroll
    for (int k = 0; k < E; ++k) {
        const float2 cs = turn ? turned[warp][j0 + k] : make_float2(1.f, 0.f);
        c[k] = cs.x, s[k] = cs.y;
    }
    const float inv_D = 1.f / (float)a.D;
    for (int h = first; h - lane / kLanes < h1; h += 2 * kHeads) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int hu = h + u * kHeads;
            const bool live = hu < h1 && in;
            float2 y[2][E / 2];  // in pairs: half the instructions
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int k = 0; k < E; k += 2) y[p][k / 2] = make_float2(x[u][p].get(k), x[u][p].get(k + 1));
            const T *weight = static_cast<const T *>(hu < a.Hq ? a.q_weight : hu < a.Hq + a.H ? a.k_weight : nullptr);
            const bool norm = live && weight != nullptr, key = hu < a.Hq + a.H;  // a query or a key
            if (a.q_weight || a.k_weight) {
                float2 squares = {0.f, 0.f};
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int k = 0; k < E / 2; ++k) squares = fma2(y[p][k], y[p][k], squares);
                float sum = squares.x + squares.y;
#pragma unroll
                for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                float f = rsqrtf(fmaf(sum, inv_D, a.eps));
                if (__any_sync(0xffffffffu, beyond_fp32(sum))) {
                    float scaled = 0.f;
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int k = 0; k < E / 2; ++k) {
                            const float v0 = y[p][k].x * kDown, v1 = y[p][k].y * kDown;
                            scaled = fmaf(v1, v1, fmaf(v0, v0, scaled));
                        }
#pragma unroll
                    for (int d = 1; d < kLanes; d <<= 1) scaled += __shfl_xor_sync(0xffffffffu, scaled, d);
                    if (norm && beyond_fp32(sum)) {
                        f = factor_beyond(scaled, inv_D, a.eps);
#pragma unroll
                        for (int p = 0; p < 2; ++p)
#pragma unroll
                            for (int k = 0; k < E / 2; ++k) y[p][k] = mul2(y[p][k], {kHalfDown, kHalfDown});
                    }
                }
                if (norm) {
                    P w[2];
                    w[0].load_shared(weight + at0);
                    w[1].load_shared(weight + at1);
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int k = 0; k < E; k += 2) y[p][k / 2] = mul2(mul2(y[p][k / 2], {f, f}), {w[p].get(k), w[p].get(k + 1)});
                }
            }
            if (live && key) {
                if (turn) {
#pragma unroll
                    for (int k = 0; k < E; k += 2) {
                        // pairs k and k + 1: elements of both pieces, or neighbours
                        const float2 c2 = {c[k], c[k + 1]}, s2 = {s[k], s[k + 1]}, less = {-s[k], -s[k + 1]};
                        if (kNeighbours) {
                            float2 &v0 = y[2 * k / E][k % (E / 2)], &v1 = y[2 * (k + 1) / E][(k + 1) % (E / 2)];
                            const float2 a0 = {v0.x, v1.x}, b0 = {v0.y, v1.y}, p0 = fma2(a0, c2, mul2(b0, less)), p1 = fma2(b0, c2, mul2(a0, s2));
                            v0 = {p0.x, p1.x};
                            v1 = {p0.y, p1.y};
                        } else {
                            const float2 b0 = y[0][k / 2], b1 = y[1][k / 2];
                            y[0][k / 2] = fma2(b0, c2, mul2(b1, less));
                            y[1][k / 2] = fma2(b1, c2, mul2(b0, s2));
                        }
                    }
                }
                if (turn || norm) {
                    x[u][0].set(y[0]);
                    x[u][1].set(y[1]);
                }
            }
            if (live) {
                T *dst = hu < a.Hq ? q_dst + hu * a.q_out_head : key ? k_dst + (hu - a.Hq) * k_step : v_dst + (hu - a.Hq - a.H) * k_step;
                x[u][0].store(dst);
                x[u][1].store(dst + apart);
            }
            fetch(hu + 2 * kHeads, x[u]);
        }
    }
}

// ---------------------------------------------------------------- any size and stride
// A warp a head, its threads pair by pair; the elements that are not rotated are pairs
// of neighbours here (the last one alone where there is an odd one).
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) rope_store_any(const __grid_constant__ Rows r) {
    const dspark_rope_store_args &a = r.a;
    after_predecessor();
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (item >= (long long)a.N * r.heads) return;
    const int i = (int)(item / r.heads), h = (int)(item - (long long)i * r.heads);
    int slot = 0;
    if (a.slot) {
        slot = checked_slot(a.slot[i], slots_of(a.n_pages, a.page), a.err);
        if (slot < 0) return;
    }
    const Head to = r.head<T>(h, i, slot);
    const T *src = static_cast<const T *>(to.src), *weight = static_cast<const T *>(to.weight);
    T *dst = static_cast<T *>(to.dst);
    float f = 1.f, down = 1.f;
    if (weight) {
        float sum = 0.f, scaled = 0.f;
        for (int d = lane; d < a.D; d += 32) {
            const float v = to_f32(src[d]), w = v * kDown;
            sum = fmaf(v, v, sum);
            scaled = fmaf(w, w, scaled);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
            scaled += __shfl_xor_sync(0xffffffffu, scaled, d);
        }
        const float inv_D = 1.f / (float)a.D;
        f = rsqrtf(fmaf(sum, inv_D, a.eps));
        if (beyond_fp32(sum)) {
            f = factor_beyond(scaled, inv_D, a.eps);
            down = kHalfDown;
        }
    }
    const int half = a.rot / 2, pos = a.pos[i];
    for (int j = lane; j < (a.D + 1) / 2; j += 32) {
        const bool turn = j < half;
        const int d0 = turn && !a.interleaved ? j : 2 * j, d1 = turn && !a.interleaved ? j + half : 2 * j + 1;
        const bool two = d1 < a.D;
        T v0 = src[d0], v1 = two ? src[d1] : v0;
        if (to.turn && (turn || weight)) {
            float b0 = to_f32(v0), b1 = to_f32(v1);
            if (weight) {
                b0 = b0 * down * f * to_f32(weight[d0]);
                if (two) b1 = b1 * down * f * to_f32(weight[d1]);
            }
            if (turn) {
                const float2 cs = cos_sin(turns_of(a.freq[j]), pos);
                const float p0 = b0;
                b0 = fmaf(p0, cs.x, -b1 * cs.y);
                b1 = fmaf(b1, cs.x, p0 * cs.y);
            }
            v0 = round_to<T>(b0);
            v1 = round_to<T>(b1);
        }
        dst[d0] = v0;
        if (two) dst[d1] = v1;
    }
}

template <typename T, int kBytes, int kLanes>
cudaError_t launch_lanes(Rows &r, cudaStream_t s) {
    constexpr int kHeads = 32 / kLanes;
    const dspark_rope_store_args &a = r.a;
    // a row's heads on one warp where there are rows enough for 16 warps an SM, else on
    // as many as that takes
    const long long want = (16ll * sm_count() + a.N - 1) / a.N;
    const int most = (r.heads + kHeads - 1) / kHeads, splits = want < 1 ? 1 : want > most ? most : (int)want;
    r.per_split = (most + splits - 1) / splits * kHeads;
    r.splits = (unsigned)((r.heads + r.per_split - 1) / r.per_split);
    const long long blocks = ((long long)a.N * r.splits + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    return a.interleaved ? launch_close(rope_store_kernel<T, kBytes, kLanes, true>, (unsigned)blocks, 32 * kWarps, 0, s, r)
                         : launch_close(rope_store_kernel<T, kBytes, kLanes, false>, (unsigned)blocks, 32 * kWarps, 0, s, r);
}

// pieces of kBytes: every address on their boundary, pairs in whole pieces
template <typename T, int kBytes>
bool fits(const dspark_rope_store_args &a, uintptr_t all) {
    constexpr int E = kBytes / (int)sizeof(T);
    const int unit = a.interleaved ? 2 * E : E;  // what rot and the rest, or their halves, consist of
    const int turned = a.interleaved ? a.rot : a.rot / 2, rest = a.interleaved ? a.D - a.rot : (a.D - a.rot) / 2;
    return all % kBytes == 0 && a.D % (2 * E) == 0 && turned % unit == 0 && rest % unit == 0 && a.D / (2 * E) <= 32;
}
template <typename T, int kBytes>
cudaError_t launch_pieces(Rows &r, cudaStream_t s) {
    const int lanes = r.a.D / (2 * (kBytes / (int)sizeof(T)));
    return lanes <= 4    ? launch_lanes<T, kBytes, 4>(r, s)
           : lanes <= 8  ? launch_lanes<T, kBytes, 8>(r, s)
           : lanes <= 16 ? launch_lanes<T, kBytes, 16>(r, s)
                         : launch_lanes<T, kBytes, 32>(r, s);
}

template <typename T>
cudaError_t launch_as(Rows &r, cudaStream_t s) {
    const dspark_rope_store_args &a = r.a;
    uintptr_t all = 0;
    auto add = [&](const void *p, int64_t row, int64_t head) {
        all |= reinterpret_cast<uintptr_t>(p) | (uintptr_t)((row | head) * (int64_t)sizeof(T));
    };
    if (a.Hq) {
        add(a.q, a.q_row, a.q_head);
        add(a.q_out, a.q_out_row, a.q_out_head);
        add(a.q_weight, 0, 0);
    }
    if (a.H) {
        add(a.k, a.k_row, a.k_head);
        add(a.k_weight, 0, 0);
        if (a.slot) {
            add(a.v, a.v_row, a.v_head);
            add(a.k_cache, a.D, 0);
            add(a.v_cache, 0, 0);
        } else {
            add(a.k_out, a.k_out_row, a.k_out_head);
        }
    }
    if (fits<T, 16>(a, all)) return launch_pieces<T, 16>(r, s);
    if (fits<T, 8>(a, all)) return launch_pieces<T, 8>(r, s);
    const long long blocks = ((long long)a.N * r.heads + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    return launch_close(rope_store_any<T>, (unsigned)blocks, 32 * kWarps, 0, s, r);
}

}  // namespace

cudaError_t launch_rope_store(const dspark_rope_store_args &a, cudaStream_t s) {
    Rows r{};
    r.a = a;
    if (!a.q) r.a.Hq = 0;
    if (!a.k) r.a.H = 0;
    r.page = page_of_size(a.slot ? a.page : 1);
    r.heads = r.a.Hq + (a.slot ? 2 : 1) * r.a.H;
    if (sm_count() < 1) return cudaErrorNoDevice;  // the work is cut by the SMs there are
    return a.dtype == DSPARK_BF16 ? launch_as<__nv_bfloat16>(r, s) : launch_as<float>(r, s);
}

}  // namespace dspark
