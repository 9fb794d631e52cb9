// attn_tc.cu -- attention of drafted rows over a paged cache on the 5th-generation
// tensor cores (bf16, D a multiple of 8 up to 128, pages of a multiple of 8 tokens).
//
// A unit's lines (rows x query heads of a group) fill one or two 128-row MMA
// operands.  Per tile of 128 tokens and operand:
//     S = Q K^T   (Q, K in shared memory, S in tensor memory, fp32)
//     P = 2^(S scale log2(e) - m)   rounded to bf16 over S's columns
//     O += P V    (P in tensor memory, V in shared memory as the MN-major operand)
// Two streams, each with its own S, O and four softmax warps, keep the tensor
// pipe and the softmax busy in turn: with two operands a stream per operand, both
// over every tile; with one, the streams take the even and the odd tiles and are
// added at the end like two partials.  Warp 8 copies keys and values by TMA, a
// box per page piece, through one ring of slots in the order of their use; warp 9
// copies Q and issues the MMAs.  The maximum m is only moved, and O rescaled in
// tensor memory, when a tile exceeds it by 2^8 (any reference gives the same
// result; P stays below 2^8 and fp32 sums far from overflow).
//
// Bound by HBM while lines are few: a tile of D = 128 is 64 KB, 2,800 clocks of an
// SM's share of the bandwidth, against about 1,050 of MMA per operand.
#include <cuda.h>
#include <cuda_bf16.h>

#include "attn_common.cuh"
#include "tc.cuh"

namespace dspark {
namespace attn {

namespace {

constexpr int kThreads = 320, kTile = 128;
constexpr float kSlack = 8.f;  // log2 by which a tile may exceed the reference

// DP: D padded to the copied width, NQ: operands a unit may have
template <int DP_, int NQ_>
struct Shape {
    static constexpr int DP = DP_, NQ = NQ_;
    static constexpr int kHalves = DP / 64;
    static constexpr int kHalf = 128 * 128;  // 128 rows of 64 bf16
    static constexpr int kSlot = kHalves * kHalf;
    static constexpr int NS = DP == 128 ? 7 - NQ : 12;  // ring slots: what 227 KB hold beside Q
    static constexpr int kOffRing = NQ * kSlot;
    static constexpr int kOffMl = kOffRing + NS * kSlot;        // float2 [2][128]
    static constexpr int kOffBar = kOffMl + 2 * 128 * 8;        // barriers
    static constexpr int kBars = 2 * NS + 9;
    static constexpr int kOffBad = kOffBar + 8 * kBars;         // uint32 [3][8]
    static constexpr int kOffMisc = kOffBad + 96;               // tmem slot, abort flag
    static constexpr int kOffScan = kOffMisc + 8;               // long long [2 + 10]
    static constexpr int kSmem = kOffScan + 96;
};

struct TcParams {
    Params p;
    int lines;  // of one operand: a whole number of rows
    int box;    // tokens of a TMA box: a power of two that divides a page
};

// A softmax warp's waits, by its first lane.  After one has run out the warp
// walks on to the end without waiting: the CTA's barriers stay paired, and the
// rows are unspecified (the error word says so).
struct Waiter {
    volatile int *abort_flag;
    int32_t *err;
    int lane;
    bool dead;
    __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity) {
        if (lane == 0 && !dead) dead = !tc::mbar_wait(bar, parity, abort_flag, err);
        __syncwarp();
    }
};

// 32 mask bits of a line from bit position pos on (its words, beyond `rows` clear)
__device__ __forceinline__ uint32_t mask_bits(const uint32_t *words, int n_words, int pos, int rows) {
    const int i = pos >> 5;
    const uint32_t lo = i < n_words ? words[i] : 0u, hi = i + 1 < n_words ? words[i + 1] : 0u;
    uint32_t v = __funnelshift_r(lo, hi, pos & 31);
    const int left = rows - pos;
    if (left <= 0) v = 0;
    else if (left < 32) v &= (1u << left) - 1;
    return v;
}

// which of the 32 tokens rel0 .. rel0 + 31 (counted from the first row of the
// cycle; negative: the cache) line `j` sees
__device__ __forceinline__ uint32_t seen_bits(const uint32_t *words, int n_words, int rel0, int rows, int j) {
    if (rel0 + 31 < 0) return 0xffffffffu;
    if (!words) {
        const int n = j - rel0 + 1;  // a chain
        return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
    }
    if (rel0 >= 0) return mask_bits(words, n_words, rel0, rows);
    return (mask_bits(words, n_words, 0, rows) << -rel0) | ((1u << -rel0) - 1);
}

template <typename C>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attention_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TcParams tp) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const Params &p = tp.p;
    const dspark_tree_attention_args &a = p.a;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar);
    uint64_t *empty = full + C::NS;
    uint64_t *s_full = empty + C::NS, *p_ready = s_full + 2, *o_done = p_ready + 2, *q_full = o_done + 2, *o_free = q_full + 1,
             *drain = o_free + 1;
    uint32_t *bad = reinterpret_cast<uint32_t *>(smem + C::kOffBad);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tc::smem_u32(smem) & 1023u) {  // the swizzled tiles need it; the launch gives it
        if (tid == 0) set_err(a.err, DSPARK_ERR_UNSUPPORTED);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < C::NS; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int w = 0; w < 2; ++w) {
            tc::mbar_init(&s_full[w], 1);
            tc::mbar_init(&p_ready[w], 4);
            tc::mbar_init(&o_done[w], 1);
        }
        tc::mbar_init(q_full, 1);
        tc::mbar_init(o_free, 8);
        tc::mbar_init(drain, 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
        p.join[blockIdx.x].pieces = 0;
    }
    if (tid < 24) bad[tid] = 0;
    if (warp == 9) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
        tc::tc_fence_before();
    }
    const Share share = share_of(p, reinterpret_cast<long long *>(smem + C::kOffScan));  // synchronises the CTA
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Walk walk(p, share);
    Piece x;

    if (warp == 8) {
        // ------------------------------------------------------------ keys and values
        uint32_t pos = 0;
        bool ok = true;
        if (lane == 0) {
            tc::prefetch_tmap(&tmK);
            tc::prefetch_tmap(&tmV);
        }
        while (ok && walk.next(x)) {
            const int32_t *table = a.table + (size_t)x.r * a.max_pages;
            const int n = x.t1 - x.t0;
            auto load = [&](const CUtensorMap *map, int t) {
                const int tok0 = t * kTile, tokens = min(kTile, x.tokens - tok0);
                const int boxes = (tokens + tp.box - 1) / tp.box;
                // a lane copies one half of one box
                const int bx = lane / C::kHalves, half = lane % C::kHalves;
                int pg = 0, off = 0;
                if (bx < boxes) {
                    const int tok = tok0 + bx * tp.box;
                    pg = table[tok / a.page];
                    off = tok % a.page;
                    if (pg < 0 || pg >= a.n_pages) {
                        set_err(a.err, DSPARK_ERR_RANGE);
                        pg = 0;
                    }
                }
                const int slot = pos % C::NS;
                int go = 1;
                if (lane == 0) {
                    go = tc::mbar_wait(&empty[slot], ((pos / C::NS) & 1u) ^ 1u, abort_flag, a.err) ? 1 : 0;
                    if (go) tc::mbar_expect_tx(&full[slot], (uint32_t)(boxes * tp.box * 128 * C::kHalves));
                }
                if (!__shfl_sync(0xffffffffu, go, 0)) return false;
                if (bx < boxes)
                    tc::tma_load_3d(smem + C::kOffRing + slot * C::kSlot + half * C::kHalf + bx * tp.box * 128, map, &full[slot],
                                    64 * half, off, pg * a.H + x.h);
                __syncwarp();
                ++pos;
                return true;
            };
            if (C::NQ == 2 && x.lines > tp.lines) {
                for (int t = x.t0; ok && t < x.t1; ++t) ok = load(&tmK, t) && load(&tmV, t);
            } else {
                ok = load(&tmK, x.t0) && (n == 1 || load(&tmK, x.t0 + 1));
                for (int t = x.t0; ok && t < x.t1; ++t) ok = load(&tmV, t) && (t + 2 >= x.t1 || load(&tmK, t + 2));
            }
        }
        if (lane == 0)  // nothing is left in flight
            for (uint32_t g = pos < (uint32_t)C::NS ? 0 : pos - C::NS; g < pos; ++g)
                tc::mbar_wait_drain(&full[g % C::NS], (g / C::NS) & 1u, a.err);
        __syncwarp();
    } else if (warp == 9) {
        // ------------------------------------------------------------ Q and the MMAs
        if (lane == 0) {
            constexpr uint32_t idesc_s = tc::idesc_bf16_f32(128, 128);
            constexpr uint32_t idesc_o = tc::idesc_bf16_f32(128, C::DP) | tc::kIdescBMnMajor;
            tc::prefetch_tmap(&tmQ);
            const uint32_t sbase = tc::smem_u32(smem);
            auto load_q = [&](const Piece &y) {
                const int ops = C::NQ == 2 && y.lines > tp.lines ? 2 : 1;
                tc::mbar_expect_tx(q_full, (uint32_t)(ops * tp.lines * 128 * C::kHalves));
                for (int o = 0; o < ops; ++o)
                    for (int half = 0; half < C::kHalves; ++half)
                        tc::tma_load_3d(smem + o * C::kSlot + half * C::kHalf, &tmQ, q_full, 64 * half, y.h * p.G,
                                        y.row0 + (y.line0 + o * tp.lines) / p.G);
            };
            uint32_t pos = 0, pieces = 0, p_count[2] = {0, 0};
            int kslot = 0, vslot = 0;
            bool more = walk.next(x), ok = true;
            uint32_t q_loads = 0;
            if (more) load_q(x), ++q_loads;
            while (ok && more) {
                const bool dual = C::NQ == 2 && x.lines > tp.lines;
                const int n = x.t1 - x.t0, steps = dual ? 2 * n : n;
                auto next_slot = [&](int &slot) {
                    slot = pos % C::NS;
                    const bool got = tc::mbar_wait(&full[slot], (pos / C::NS) & 1u, abort_flag, a.err);
                    ++pos;
                    return got;
                };
                auto scores = [&](int i) {
                    const int w = i & 1;
                    if ((!dual || w == 0) && !next_slot(kslot)) return false;
                    tc::tc_fence_after();
                    const uint64_t ad = tc::smem_desc_k128(sbase + (dual && w ? C::kSlot : 0));
                    const uint64_t bd = tc::smem_desc_k128(sbase + C::kOffRing + kslot * C::kSlot);
#pragma unroll
                    for (int kk = 0; kk < C::DP / 16; ++kk) {
                        const uint64_t step = (uint64_t)(((kk >> 2) * C::kHalf + (kk & 3) * 32) >> 4);
                        tc::umma_bf16(tmem + 128 * w, ad + step, bd + step, idesc_s, kk > 0 ? 1u : 0u);
                    }
                    tc::umma_commit(&s_full[w]);
                    if (!dual || w == 1) tc::umma_commit(&empty[kslot]);
                    return true;
                };
                ok = tc::mbar_wait(q_full, pieces & 1u, abort_flag, a.err);
                ok = ok && scores(0) && (steps == 1 || scores(1));
                for (int i = 0; ok && i < steps; ++i) {
                    const int w = i & 1;
                    ok = tc::mbar_wait(&p_ready[w], p_count[w]++ & 1u, abort_flag, a.err);
                    if (ok && i == 0 && pieces > 0) ok = tc::mbar_wait(o_free, (pieces - 1) & 1u, abort_flag, a.err);
                    if (!ok) break;
                    if (i == steps - 1) {  // every S of the piece is done: Q may go
                        more = walk.next(x);
                        if (more) load_q(x), ++q_loads;
                    }
                    if ((!dual || w == 0) && !next_slot(vslot)) {
                        ok = false;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint64_t bd = tc::smem_desc_mn128(sbase + C::kOffRing + vslot * C::kSlot, C::kHalf);
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        tc::umma_bf16_ta(tmem + 256 + 128 * w, tmem + 128 * w + 8 * kk, bd + (uint64_t)((kk * 2048) >> 4),
                                         idesc_o, i >= 2 || kk > 0 ? 1u : 0u);
                    tc::umma_commit(&o_done[w]);
                    if (!dual || w == 1) tc::umma_commit(&empty[vslot]);
                    if (i + 2 < steps) ok = scores(i + 2);
                }
                ++pieces;
            }
            if (!ok) {
                // given up: let what was issued finish before memory is released
                if (q_loads) tc::mbar_wait_drain(q_full, (q_loads - 1) & 1u, a.err);
                tc::umma_commit(drain);
                tc::mbar_wait_drain(drain, 0u, a.err);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int w = warp >> 2, q = warp & 3, row = 32 * q + lane;
        const uint32_t quad = (uint32_t)(32 * q) << 16;
        const uint32_t s_tmem = tmem + quad + 128 * w;
        float2 *ml = reinterpret_cast<float2 *>(smem + C::kOffMl);
        Waiter wait{abort_flag, a.err, lane, false};
        uint32_t s_count = 0, done0 = 0, done1 = 0, base = 0, pieces = 0;
        const float scale = fmaxf(fabsf(p.scale_log2), 1e-37f);
        while (walk.next(x)) {
            const bool dual = C::NQ == 2 && x.lines > tp.lines;
            const int n = x.t1 - x.t0;
            const int lines = dual ? (w ? x.lines - tp.lines : tp.lines) : x.lines;
            const int steps = dual ? n : (n + 1 - w) >> 1;
            const int line = x.line0 + (dual && w ? tp.lines : 0) + row;
            const bool active = 32 * q < lines, live = row < lines;
            const int j = line / p.G;
            // rows of the cycle before `base_rel` are seen by every line of the unit
            const int base_rel = a.mask ? 0 : x.line0 / p.G + 1;
            const uint32_t *words = a.mask && live ? reinterpret_cast<const uint32_t *>(a.mask + (size_t)(x.row0 + j) * a.W) : nullptr;
            uint32_t *flags = bad + 8 * (pieces % 3u);
            float m = -INFINITY, l = 0.f;
            for (int k = 0; k < steps; ++k) {
                const int t = dual ? x.t0 + k : x.t0 + 2 * k + w;
                const int tok0 = t * kTile;
                const bool tail = tok0 + kTile > x.len + base_rel;
                if (tail && (!dual || w == 0)) {
                    // Values that some lines do not see must not reach them as 0 x inf:
                    // slots beyond the tokens are zeroed, infinities and NaN of the
                    // cycle's rows too, and those added back below where they are seen.
                    const int tl = t - x.t0;
                    const uint32_t pos = base + (uint32_t)(dual ? 2 * tl + 1 : tl + min(tl + 2, n));
                    const int slot = pos % C::NS;
                    wait(&full[slot], (pos / C::NS) & 1u);
                    const int tok = tok0 + row, rel = tok - x.len - base_rel;
                    if (tok >= x.tokens || rel >= 0) {
                        bool found = false;
#pragma unroll 1
                        for (int c = 0; c < 8 * C::kHalves; ++c) {
                            uint4 *at = reinterpret_cast<uint4 *>(smem + C::kOffRing + slot * C::kSlot + (c >> 3) * C::kHalf +
                                                                  row * 128 + ((c + lane) & 7) * 16);
                            if (tok >= x.tokens) {
                                *at = make_uint4(0u, 0u, 0u, 0u);
                                continue;
                            }
                            uint4 v = *at;
                            uint32_t e[4] = {v.x, v.y, v.z, v.w};
                            bool hit = false;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if ((e[i] & 0x7f80u) == 0x7f80u) e[i] &= 0xffff0000u, hit = true;
                                if ((e[i] & 0x7f800000u) == 0x7f800000u) e[i] &= 0xffffu, hit = true;
                            }
                            if (hit) {
                                *at = make_uint4(e[0], e[1], e[2], e[3]);
                                found = true;
                            }
                        }
                        if (found && rel < 256) atomicOr(&flags[rel >> 5], 1u << (rel & 31));
                        tc::fence_proxy_async_smem();
                    }
                }
                wait(&s_full[w], s_count++ & 1u);
                tc::tc_fence_after();
                if (active) {
                    float s[128];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tc::tmem_ld32(s_tmem + 32 * c, s + 32 * c);
                    tc::tmem_wait_ld();
                    if (p.scale_log2 < 0.f) {
#pragma unroll
                        for (int i = 0; i < 128; ++i) s[i] = -s[i];
                    }
                    if (tail) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int rel0 = tok0 + 32 * c - x.len;
                            // lines beyond the unit's see nothing; what they hold is not read
                            const uint32_t see = live ? seen_bits(words, 2 * a.W, rel0, x.rows, j) : 0u;
#pragma unroll
                            for (int i = 0; i < 32; ++i) s[32 * c + i] = (see >> i) & 1u ? s[32 * c + i] : -INFINITY;
                        }
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 128; i += 4)
#pragma unroll
                        for (int c = 0; c < 4; ++c) mx[c] = fmaxf(mx[c], s[i + c]);
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
                    if (k == 0) {
                        m = top;
                    } else if (__any_sync(0xffffffffu, top > m + kSlack)) {
                        const float to = top > m + kSlack ? top : m;
                        const float f = to == -INFINITY ? 1.f : ex2(m - to);
                        m = to;
                        l *= f;
                        wait(&o_done[w], ((w ? done1 : done0) + k - 1) & 1u);
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < C::DP; c += 32) {
                            float o[32];
                            tc::tmem_ld32(tmem + quad + 256 + 128 * w + c, o);
                            tc::tmem_wait_ld();
                            uint32_t r[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(o[i] * f);
                            tc::tmem_st32(tmem + quad + 256 + 128 * w + c, r);
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : m;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t r[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float p0 = ex2(fmaf(s[64 * c + 2 * i], scale, -ref));
                            const float p1 = ex2(fmaf(s[64 * c + 2 * i + 1], scale, -ref));
                            sum[i & 3] += p0 + p1;
                            const __nv_bfloat162 two = __floats2bfloat162_rn(p0, p1);
                            r[i] = *reinterpret_cast<const uint32_t *>(&two);
                        }
                        tc::tmem_st32(s_tmem + 32 * c, r);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&p_ready[w]);
            }

            // ---------------------------------------------------------- the piece's end
            const bool two = !dual && n > 1;  // both streams hold a part of the same lines
            if (two) ml[128 * w + row] = make_float2(m, l);
            if (tid < 8) bad[8 * ((pieces + 1) % 3u) + tid] = 0;
            tc::named_bar_sync(1, 256);
            float M = m, f0 = 1.f, f1 = 0.f;
            if (!dual) {
                const float2 s0 = two ? ml[row] : make_float2(m, l), s1 = two ? ml[128 + row] : make_float2(-INFINITY, 0.f);
                if (two) {
                    M = fmaxf(s0.x, s1.x);
                    const float ref = M == -INFINITY ? 0.f : M;
                    f0 = ex2(s0.x - ref);
                    f1 = ex2(s1.x - ref);
                    l = fmaf(f0, s0.y, f1 * s1.y);
                }  // else the only tile was stream 0's, and its warps finish the lines alone
            }
            const uint32_t steps0 = dual ? n : (n + 1) >> 1, steps1 = dual ? n : n >> 1;
            if (!dual || w == 0) wait(&o_done[0], (done0 + steps0 - 1) & 1u);
            if (steps1 > 0 && (!dual || w == 1)) wait(&o_done[1], (done1 + steps1 - 1) & 1u);
            tc::tc_fence_after();
            if (two) tc::named_bar_sync(1, 256);  // ml has been read
            uint32_t any_bad = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) any_bad |= flags[i];
            if (active && (dual || two || w == 0)) {
                const int unit_line = line - x.line0;
                const float inv = x.slot < 0 ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                const size_t orow = (size_t)(x.row0 + j) * a.Hq + x.h * p.G + line % p.G;
                const size_t prow = (size_t)(x.slot < 0 ? 0 : x.slot) * p.block + unit_line;
                // with two streams of the same lines each takes half of the columns
                const int c0 = two ? w * (C::DP / 2) : 0, c1 = two ? c0 + C::DP / 2 : C::DP;
#pragma unroll 1
                for (int c = c0; c < c1; c += 32) {
                    float o[32];
                    tc::tmem_ld32(tmem + quad + 256 + (dual ? 128 * w : 0) + c, o);
                    if (two) {
                        float o1[32];
                        tc::tmem_ld32(tmem + quad + 384 + c, o1);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = fmaf(f0, o[i], f1 * o1[i]);
                    } else {
                        tc::tmem_wait_ld();
                    }
                    if (any_bad && live) {
                        for (int b = 0; b < 256; ++b) {
                            if (!((flags[b >> 5] >> (b & 31)) & 1u)) continue;
                            const int rel = b + base_rel, tok = x.len + rel;
                            if (!(seen_bits(words, 2 * a.W, rel, x.rows, j) & 1u)) continue;
                            int pg = a.table[(size_t)x.r * a.max_pages + tok / a.page];
                            if (pg < 0 || pg >= a.n_pages) pg = 0;
                            const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v_cache) +
                                                     (((size_t)pg * a.H + x.h) * a.page + tok % a.page) * a.D + c;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                if (c + i >= a.D) break;
                                const float e = __bfloat162float(v[i]);
                                if (!(fabsf(e) < INFINITY)) o[i] += e;
                            }
                        }
                    }
                    if (!live) continue;
                    if (x.slot < 0) {
                        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + orow * a.D + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            if (c + i >= a.D) break;
                            uint32_t r[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 v = __floats2bfloat162_rn(o[i + 2 * e] * inv, o[i + 2 * e + 1] * inv);
                                r[e] = *reinterpret_cast<const uint32_t *>(&v);
                            }
                            *reinterpret_cast<uint4 *>(out + i) = make_uint4(r[0], r[1], r[2], r[3]);
                        }
                    } else {
                        float *out = p.part_o + prow * a.D + c;
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            if (c + i >= a.D) break;
                            *reinterpret_cast<float4 *>(out + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        }
                    }
                }
                if (live && (dual || w == 0)) {
                    if (x.slot >= 0) p.part_ml[prow] = make_float2(M, l);
                    else if (a.lse) a.lse[orow] = lse_of(M, l);
                }
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(o_free);
            if (tid == 0 && x.t0 == 0 && x.t1 < x.tiles) p.join[blockIdx.x] = walk.join_of(x);
            done0 += steps0;
            done1 += steps1;
            base += 2 * (uint32_t)n;
            ++pieces;
        }
        tc::tc_fence_before();
    }
    __syncthreads();
    if (warp == 9) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// a map of the cache as [n_pages H][page][D], boxes of 64 columns x box tokens
bool encode_cache(CUtensorMap *m, const void *base, const dspark_tree_attention_args &a, int box) {
    const uint64_t dims[3] = {(uint64_t)a.D, (uint64_t)a.page, (uint64_t)a.n_pages * a.H};
    const uint64_t strides[2] = {(uint64_t)a.D * 2, (uint64_t)a.page * a.D * 2};
    const uint32_t bx[3] = {64, (uint32_t)box, 1};
    return encode_bf16_map3(m, base, dims, strides, bx);
}

template <typename C>
cudaError_t launch_as(const TcParams &tp, int grid, const CUtensorMap &q, const CUtensorMap &k, const CUtensorMap &v,
                      cudaStream_t s) {
    auto kern = tree_attention_tc<C>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    kern<<<grid, kThreads, C::kSmem, s>>>(q, k, v, tp);
    return cudaGetLastError();
}

// lines of one operand: whole rows of a group's query heads
int lines_of(const dspark_tree_attention_args &a) {
    const int G = a.Hq / a.H;
    return 128 / G * G;
}

}  // namespace

bool tc_supported(const dspark_tree_attention_args &a) {
    auto al16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
    return a.dtype == DSPARK_BF16 && a.D % 8 == 0 && a.D <= 128 && a.page % 8 == 0 && a.Hq / a.H <= 128 && al16(a.q) &&
           al16(a.k_cache) && al16(a.v_cache) && al16(a.out) && a.q_row % 8 == 0 && a.q_head % 8 == 0 && a.q_row > 0 &&
           a.q_head > 0 && a.q_row < (1ll << 38) && tc_kernels_enabled() && tc_available();
}

int tc_block(const dspark_tree_attention_args &a) {
    const long long most = (long long)a.max_rows * (a.Hq / a.H);
    return lines_of(a) * (most > lines_of(a) ? 2 : 1);
}

cudaError_t launch_tc(Params p, int grid, cudaStream_t s) {
    const dspark_tree_attention_args &a = p.a;
    TcParams tp{};
    tp.lines = lines_of(a);
    p.tile = kTile;
    tp.p = p;
    tp.box = a.page & -a.page;
    if (tp.box > kTile) tp.box = kTile;
    CUtensorMap q, k, v;
    const uint64_t dims[3] = {(uint64_t)a.D, (uint64_t)a.Hq, (uint64_t)a.N};
    const uint64_t strides[2] = {(uint64_t)a.q_head * 2, (uint64_t)a.q_row * 2};
    const uint32_t bx[3] = {64, (uint32_t)p.G, (uint32_t)(tp.lines / p.G)};
    if (!encode_bf16_map3(&q, a.q, dims, strides, bx) || !encode_cache(&k, a.k_cache, a, tp.box) ||
        !encode_cache(&v, a.v_cache, a, tp.box))
        return cudaErrorInvalidValue;
    const bool two = p.block > tp.lines;
    if (a.D > 64)
        return two ? launch_as<Shape<128, 2>>(tp, grid, q, k, v, s) : launch_as<Shape<128, 1>>(tp, grid, q, k, v, s);
    return two ? launch_as<Shape<64, 2>>(tp, grid, q, k, v, s) : launch_as<Shape<64, 1>>(tp, grid, q, k, v, s);
}

}  // namespace attn
}  // namespace dspark
