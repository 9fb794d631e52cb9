// attn4_mma.cu -- attention of few lines over a cache in 4 bits: values unpacked in
// registers, products by the warp's own matrix instructions.
//
// While a unit has few lines the cache is read for few products, and what counts is how
// a tile gets from 4 bits to the tensor cores.  Through shared memory as 16-bit tiles (the
// kernel of attn4_tc.cu) a tile of 128 tokens is written and read back as 64 KB, and its two
// products take 128 rows however few are in use.  Here nothing of it goes back to
// shared memory: the fragments of an m16n8k16 product are unpacked where they are used.
//
// A unit's lines (rows x query heads of a group) are MT times 16.  A producer warp walks the
// CTA's share and copies tiles into a ring of steps of 32 tokens (codes and scales of
// keys and values, bulk copies of a page piece each); warp w of NW takes every NW-th step,
// with a running maximum and sum and 16 MT x D sums of its own, and the warps' results are
// added at the piece's end like partials.  Per step and warp:
//     S = Q K^T          K in bf16 (exactly), contracted over D in an order of its own:
//                        lane j of four has columns j D/4 .. of a token, 16 adjacent bytes
//     P = 2^(S scale log2(e) - m), rounded to fp16; m moves when a weight would pass 2^15
//     O += P V           V in fp16 as eighths (exactly), column n of the i-th product of a
//                        token is element i of its n-th group, 8 adjacent bytes
// A product's columns are tokens in the order 0 4 1 5 2 6 3 7, so that the rows of values that
// four lanes read are adjacent, and both reads are free of bank conflicts.
//
// Instructions of a tile of 128 tokens x 128, keys and values: 1.4 per element of keys, 1.75
// per element of values to unpack, 256 MT matrix products.
#include "attn_tc_kernel.cuh"

namespace dspark {
namespace attn {

namespace {

constexpr int kStep = 32;     // tokens of a step
constexpr float kLift = 7.f;  // the reference stands below the maximum, as in attn_tc_kernel.cuh
constexpr int kMmaUnitCost = 4;

template <int DP_, int MT_>
struct MmaShape {
    static constexpr int DP = DP_, MT = MT_;
    // with the producer 12 warps of 168 registers, or 8 of 255
    static constexpr int NW = MT == 1 ? 11 : 7, kThreads = 32 * (NW + 1);
    static constexpr int kLines = 16 * MT;
    static constexpr int NS = 2 * NW;                  // ring slots: a step each, always of the same warp
    static constexpr int kSlot = kStep * DP / 16 * 18;  // codes of keys, of values, scales of keys, of values
    static constexpr int kOffO = NS * kSlot;            // float [NW][kLines][DP]
    static constexpr int kOffQ = kOffO + NW * kLines * DP * 4;  // uint4 [MT][DP / 16][32]
    static constexpr int kOffMl = kOffQ + MT * DP / 16 * 512;   // float2 [NW][kLines]
    static constexpr int kOffPiece = kOffMl + NW * kLines * 8;
    static constexpr int kOffBar = kOffPiece + 64 * kQueue;
    static constexpr int kOffMisc = kOffBar + 8 * (2 * NS + 2 * kQueue);
    static constexpr int kSmem = kOffMisc + 8;
    static_assert(kSlot % 16 == 0 && kOffPiece % 16 == 0, "places");
};

struct MmaParams {
    Params p;
    int box;  // tokens of a copy
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// a barrier of the consuming warps; true where any of them says so
__device__ __forceinline__ bool meet(int threads, bool any) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"(any ? 1u : 0u), "r"(threads)
        : "memory");
    return r != 0;
}

// Two values n s of bf16 from nibble p of a word's halves: 128 + (n + 8) by its bits, times s,
// minus 136 s (17 s 8: eight bits, nothing is rounded).
__device__ __forceinline__ uint32_t keys_of(uint32_t word, int p, const __nv_bfloat162 &s, const __nv_bfloat162 &off) {
    const uint32_t v = ((word >> (4 * p)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 y = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v), s, off);
    return *reinterpret_cast<const uint32_t *>(&y);
}
// Two values n s of fp16: 1024 + (n + 8), or 1024 + 16 (n + 8) one nibble up, to n, times s
__device__ __forceinline__ uint32_t values_of(uint32_t word, int odd, const __half2 &s) {
    __half2 n;
    if (odd) {
        const uint32_t v = (word & 0x00f000f0u) | 0x64006400u;
        n = __hfma2(*reinterpret_cast<const __half2 *>(&v), __floats2half2_rn(0.0625f, 0.0625f), __floats2half2_rn(-72.f, -72.f));
    } else {
        const uint32_t v = (word & 0x000f000fu) | 0x64006400u;
        n = __hadd2(*reinterpret_cast<const __half2 *>(&v), __floats2half2_rn(-1032.f, -1032.f));
    }
    const __half2 y = __hmul2(n, s);
    return *reinterpret_cast<const uint32_t *>(&y);
}
__device__ __forceinline__ float eighth_of(unsigned b) {  // s(b) / 8
    return b == cache4::kNoNumbers ? __uint_as_float(0x7fc00000u) : __uint_as_float((b + (108u << 3)) << 20);
}

// steps of a piece
__device__ __forceinline__ int steps_of(const Piece &x) {
    return (min(x.t1 << kTileLog2, x.tokens) - (x.t0 << kTileLog2) + kStep - 1) / kStep;
}

// ---------------------------------------------------------------- the producer
template <typename C>
__device__ __forceinline__ void produce(unsigned char *smem, const MmaParams &mp, const Waiter &wait, uint64_t *full, uint64_t *empty,
                                        uint64_t *queue_full, uint64_t *queue_empty) {
    const Params &p = mp.p;
    const dspark_tree_attention_args &a = p.a;
    const int lane = threadIdx.x & 31, box = mp.box, boxes_step = kStep / box;
    const int code_row = a.D / 2, scale_row = a.D / 16;
    const long long page_bytes = cache4::page_bytes(a.page, a.D), codes = cache4::code_bytes(a.page, a.D);
    const Share share = share_of(p);
    Walk walk(p, share);
    if (lane == 0) p.join[blockIdx.x].pieces = 0;
    Piece x;
    uint32_t c = 0;  // steps handed out
    bool more = true, ok = true;
    for (uint32_t k = 0; more && ok; ++k) {
        more = walk.next(x);
        if (!more) x.r = -1;
        const int qi = k % kQueue;
        ok = wait.warp(&queue_empty[qi], ((k / kQueue) & 1u) ^ 1u);
        if (!ok) break;
        if (lane == 0) {
            *reinterpret_cast<Piece *>(smem + C::kOffPiece + 64 * qi) = x;
            tc::mbar_arrive(&queue_full[qi]);
            if (more && x.t0 == 0 && x.t1 < x.tiles) p.join[blockIdx.x] = walk.join_of(x);
        }
        if (!more) break;
        const int32_t *table = a.table + (size_t)x.r * a.max_pages;
        const int last = x.tokens - 1, h = x.head / p.subs;
        int in_table = 0;  // of this lane's box
        auto page_at = [&](int t) { return table[in_table = p.page.of(lookup_token(t, kTileLog2, lane, box, last))]; };
        int pg = page_at(x.t0);
        for (int t = x.t0; t < x.t1; ++t) {
            const int tok0 = t << kTileLog2, here = min(kTile, x.tokens - tok0);
            const int boxes = (here + box - 1) / box, steps = (here + kStep - 1) / kStep;
            const bool mine = lane < steps;
            const uint32_t s = c + lane;
            bool got = true;
            if (mine) got = wait.one(&empty[s % C::NS], ((s / C::NS) & 1u) ^ 1u);
            ok = __all_sync(0xffffffffu, got);
            if (!ok) break;
            if (mine) tc::mbar_expect_tx(&full[s % C::NS], (uint32_t)(min(boxes - lane * boxes_step, boxes_step) * box * scale_row * 18));
            __syncwarp();
            if (lane < boxes && (pg < 0 || pg >= a.n_pages)) {
                set_err(a.err, DSPARK_ERR_RANGE);
                pg = 0;
            }
            const long long at_page = ((long long)pg * a.H + h) * page_bytes;
            const int off = tok0 + lane * box - in_table * a.page;  // of the lane's box in its page
            // box i / 4: codes of keys, of values, scales of keys, of values
            for (int i0 = 0; i0 < 4 * boxes; i0 += 32) {
                const int i = i0 + lane, b = i >> 2;
                const long long from_page = __shfl_sync(0xffffffffu, at_page, b & 31);
                const int from = __shfl_sync(0xffffffffu, off, b & 31);
                if (i < 4 * boxes) {
                    const bool values = i & 1, scales = i & 2;
                    const int row = scales ? scale_row : code_row, step = b / boxes_step;
                    const unsigned char *src = static_cast<const unsigned char *>(values ? a.v_cache : a.k_cache) + from_page +
                                               (scales ? codes : 0) + (long long)from * row;
                    const uint32_t slot = (c + step) % C::NS;
                    unsigned char *dst = smem + slot * C::kSlot + (scales ? 2 * kStep * code_row : 0) + (values ? kStep * row : 0) +
                                         (b - step * boxes_step) * box * row;
                    tc::bulk_load(dst, src, (uint32_t)(box * row), &full[slot]);
                }
            }
            c += steps;
            if (t + 1 < x.t1) pg = page_at(t + 1);
        }
    }
    __syncwarp();
    if (*wait.abort_flag) {
        // given up: let the copies land before the CTA's memory goes
        for (uint32_t k = lane; k < (uint32_t)C::NS; k += 32)
            if (k < c) tc::mbar_wait_drain(&full[(c - 1 - k) % C::NS], ((c - 1 - k) / C::NS) & 1u, a.err);
    }
}

// ---------------------------------------------------------------- the consumers
// the queries of a unit as fragments of the first product, zero beyond its lines and columns
template <typename C>
__device__ __forceinline__ void load_queries(unsigned char *smem, const Params &p, const Piece &x) {
    constexpr int kParts = C::DP / 4, kLane = C::DP / 4;  // parts of 4 elements of a line; columns of a lane
    const dspark_tree_attention_args &a = p.a;
    const int h = x.head / p.subs, sub = x.head - h * p.subs;
    const int head0 = h * p.G + sub * p.heads, heads = min(p.heads, p.G - sub * p.heads);
    uint32_t *q = reinterpret_cast<uint32_t *>(smem + C::kOffQ);
    for (int i = threadIdx.x; i < C::kLines * kParts; i += 32 * C::NW) {
        const int line = i / kParts, d = (i % kParts) * 4, jj = line / p.heads, g = line - jj * p.heads;
        uint2 v = make_uint2(0u, 0u);
        if (jj < x.n && g < heads && d < a.D)
            v = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.q) + (long long)(x.row0 + x.first + jj) * a.q_row +
                                                 (head0 + g) * a.q_head + d);
        const int m = line >> 4, r = line & 7, up = (line >> 3) & 1, j = d / kLane, ks = (d % kLane) / 4;
        uint32_t *to = q + ((m * (C::DP / 16) + ks) * 32 + r * 4 + j) * 4 + up;
        to[0] = v.x;
        to[2] = v.y;
    }
}

template <typename C, bool kRows16>  // kRows16: a token's codes start on 16 bytes
__device__ __forceinline__ void consume(unsigned char *smem, const MmaParams &mp, const Waiter &wait, uint64_t *full, uint64_t *empty,
                                        uint64_t *queue_full, uint64_t *queue_empty) {
    constexpr int DP = C::DP, MT = C::MT, KS = DP / 16, ND = DP / 8;
    const Params &p = mp.p;
    const dspark_tree_attention_args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    const int code_row = a.D / 2, scale_row = a.D / 16;
    const float scale = fmaxf(p.scale_log2, 1e-37f);  // 0 would make -inf x 0 of what is not seen
    const int token_k = (r >> 1) + 4 * (r & 1);        // token of a product's column r
    const uint4 *q = reinterpret_cast<const uint4 *>(smem + C::kOffQ) + lane;
    float *part = reinterpret_cast<float *>(smem + C::kOffO);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::kOffMl);
    Queue queue{reinterpret_cast<const Piece *>(smem + C::kOffPiece), queue_full, queue_empty, 0};
    auto next_piece = [&](Piece &x) {
        const int i = queue.n % kQueue;
        if (!wait.warp(&queue_full[i], (queue.n / kQueue) & 1u)) return false;
        x = *reinterpret_cast<const Piece *>(smem + C::kOffPiece + 64 * i);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&queue_empty[i]);
        ++queue.n;
        return true;
    };
    Piece x;
    bool ok = next_piece(x);
    if (!ok) x.r = -1;
    if (x.r >= 0) load_queries<C>(smem, p, x);
    if (meet(32 * C::NW, !ok)) return;
    uint32_t c0 = 0;  // steps before the piece
    while (x.r >= 0) {
        const int steps = steps_of(x);
        // this warp's lines r, r + 8 (+ 16 m) as rows of the request
        const int base_rel = a.mask ? 0 : x.first + 1;  // rows of the cycle before it are seen by every line
        float O[MT][ND][4], m[MT][2], l[MT][2];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int n = 0; n < ND; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) O[t][n][e] = 0.f;
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
        }
        const uint32_t skip = (warp + C::NW - c0 % C::NW) % C::NW;
#pragma unroll 1
        for (int s = skip; s < steps; s += C::NW) {
            const uint32_t c = c0 + s;
            const int slot = c % C::NS, tok0 = (x.t0 << kTileLog2) + s * kStep;
            ok = wait.warp(&full[slot], (c / C::NS) & 1u);
            if (!ok) break;
            const unsigned char *kcode = smem + slot * C::kSlot, *vcode = kcode + kStep * code_row, *kscale = vcode + kStep * code_row,
                                *vscale = kscale + kStep * scale_row;
            const bool tail = tok0 + kStep > x.len + base_rel;
            // ------------------------------------------------ S = Q K^T
            float S[MT][4][4];
            uint32_t kw[4][KS / 2];
            __nv_bfloat162 ks[4][KS / 4], koff[4][KS / 4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int tok = 8 * t + token_k;
                const unsigned char *at = kcode + tok * code_row + j * (DP / 8), *sc = kscale + tok * scale_row + j * (DP / 64);
                if (kRows16 && DP == 128) {
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (32 * j < a.D) w = *reinterpret_cast<const uint4 *>(at);
                    kw[t][0] = w.x, kw[t][1] = w.y, kw[t][KS / 2 - 2] = w.z, kw[t][KS / 2 - 1] = w.w;
                } else {
#pragma unroll
                    for (int g = 0; g < KS / 4; ++g) {
                        uint2 w = make_uint2(0u, 0u);
                        if (j * (DP / 4) + 16 * g < a.D) w = *reinterpret_cast<const uint2 *>(at + 8 * g);
                        kw[t][2 * g] = w.x, kw[t][2 * g + 1] = w.y;
                    }
                }
#pragma unroll
                for (int g = 0; g < KS / 4; ++g) {
                    uint32_t s1 = 0;
                    if (j * (DP / 4) + 16 * g < a.D) {
                        const uint32_t b = sc[g];
                        s1 = b == cache4::kNoNumbers ? 0x7fc0u : (b + (111u << 3)) << 4;
                    }
                    const uint32_t s2 = s1 * 0x10001u;
                    ks[t][g] = *reinterpret_cast<const __nv_bfloat162 *>(&s2);
                    koff[t][g] = __hmul2(ks[t][g], __floats2bfloat162_rn(-136.f, -136.f));
                }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[i][t][e] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint4 qa[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) qa[i] = q[(i * KS + k) * 32];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t b0 = keys_of(kw[t][k >> 1], 2 * (k & 1), ks[t][k >> 2], koff[t][k >> 2]);
                    const uint32_t b1 = keys_of(kw[t][k >> 1], 2 * (k & 1) + 1, ks[t][k >> 2], koff[t][k >> 2]);
#pragma unroll
                    for (int i = 0; i < MT; ++i) mma_bf16(S[i][t], qa[i], b0, b1);
                }
            }
            // ------------------------------------------------ the values' words, and the slot is free
            uint32_t vw[2][4][ND / 8], vs[2][4];
#pragma unroll
            for (int kc = 0; kc < 2; ++kc)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int tok = 16 * kc + 4 * e + j;
                    const bool in = r * ND < a.D;
                    const unsigned char *at = vcode + tok * code_row + r * (ND / 2);
                    vs[kc][e] = 0;
                    if (DP == 128) {
                        uint2 w = make_uint2(0u, 0u);
                        if (in) w = *reinterpret_cast<const uint2 *>(at);
                        vw[kc][e][0] = w.x, vw[kc][e][ND / 8 - 1] = w.y;
                    } else {
                        vw[kc][e][0] = in ? *reinterpret_cast<const uint32_t *>(at) : 0u;
                    }
                    if (in) vs[kc][e] = vscale[tok * scale_row + r * ND / 16];
                }
            uint32_t no_numbers[2] = {0u, 0u};  // tokens of this step whose groups 2 j, 2 j + 1 (of ND columns) are NaN for those who see them
            if (tail) {
                // what some lines do not see must not reach them as 0 x NaN: it counts as zeros here, and
                // the lines that do see it are told below
#pragma unroll 1
                for (int i = 0; i < kStep; ++i) {
                    const int rel = tok0 + i - x.len;
                    if (rel < base_rel || tok0 + i >= x.tokens) continue;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int d = (2 * j + g) * ND;
                        if (d < a.D && vscale[i * scale_row + d / 16] == cache4::kNoNumbers) no_numbers[g] |= 1u << i;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&empty[slot]);
            // ------------------------------------------------ the weights
            uint32_t see[MT][2];
            if (tail) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int line = 16 * i + 8 * u + r, jj = line / p.heads, row = x.first + jj;
                        see[i][u] = 0;
                        if (jj < x.n) {
                            const uint32_t *words = a.mask ? reinterpret_cast<const uint32_t *>(a.mask + (size_t)(x.row0 + row) * a.W) : nullptr;
                            see[i][u] = seen_bits(words, 2 * a.W, tok0 - x.len, x.rows, row);
                        }
                    }
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!((see[i][e >> 1] >> (8 * t + j + 4 * (e & 1))) & 1u)) S[i][t][e] = -INFINITY;
            }
            float top[MT][2];
            bool over = false;
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float v = -INFINITY;
#pragma unroll
                    for (int t = 0; t < 4; ++t) v = fmaxf(v, fmaxf(S[i][t][2 * u], S[i][t][2 * u + 1]));
                    top[i][u] = v * scale;
                    over |= top[i][u] > m[i][u] + (kLift + kSlack);
                }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    float f[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float v = top[i][u];
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                        const float to = v > m[i][u] + (kLift + kSlack) ? v - kLift : m[i][u];
                        f[u] = to == -INFINITY ? 1.f : ex2(m[i][u] - to);
                        m[i][u] = to;
                        l[i][u] *= f[u];
                    }
#pragma unroll
                    for (int n = 0; n < ND; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) O[i][n][e] *= f[e >> 1];
                }
            }
            uint32_t P[MT][4][2];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float ref = m[i][u] == -INFINITY ? 0.f : m[i][u];
                    const float2 by = {scale, scale}, off = {-ref, -ref};
                    float2 sum = {0.f, 0.f};
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const float2 arg = fma2({S[i][t][2 * u], S[i][t][2 * u + 1]}, by, off);
                        const float2 e = {ex2(arg.x), ex2(arg.y)};
                        sum = add2(sum, e);
                        P[i][t][u] = pack_half(e.x, e.y);
                    }
                    l[i][u] += sum.x + sum.y;
                }
            // ------------------------------------------------ O += P V
#pragma unroll
            for (int kc = 0; kc < 2; ++kc) {
                __half2 sv[2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t b = vs[kc][2 * half + e];
                        f[e] = eighth_of(b);
                        if (tail) {
                            const int tok = tok0 + 16 * kc + 8 * half + 4 * e + j;
                            if (tok >= x.tokens || (b == cache4::kNoNumbers && tok - x.len >= base_rel)) f[e] = 0.f;
                        }
                    }
                    sv[half] = __floats2half2_rn(f[0], f[1]);
                }
                uint32_t pa[MT][4];
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    pa[i][0] = P[i][2 * kc][0], pa[i][1] = P[i][2 * kc][1], pa[i][2] = P[i][2 * kc + 1][0], pa[i][3] = P[i][2 * kc + 1][1];
#pragma unroll
                for (int w = 0; w < ND / 8; ++w) {
                    // the elements of even and of odd places of two tokens side by side, for either half of the 16
                    uint32_t two[2][2];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        two[half][0] = __byte_perm(vw[kc][2 * half][w], vw[kc][2 * half + 1][w], 0x5410);
                        two[half][1] = __byte_perm(vw[kc][2 * half][w], vw[kc][2 * half + 1][w], 0x7632);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int sh = 8 * (e >> 2), odd = (e >> 1) & 1;
                        const uint32_t b0 = values_of(two[0][e & 1] >> sh, odd, sv[0]), b1 = values_of(two[1][e & 1] >> sh, odd, sv[1]);
#pragma unroll
                        for (int i = 0; i < MT; ++i) mma_f16(O[i][8 * w + e], pa[i], b0, b1);
                    }
                }
            }
            if (tail && (no_numbers[0] | no_numbers[1])) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (see[i][e >> 1] & no_numbers[e & 1]) {
#pragma unroll
                            for (int n = 0; n < ND; ++n) O[i][n][e] = NAN;
                        }
            }
        }
        c0 += (uint32_t)steps;

        // ---------------------------------------------------- the piece's end
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float v = l[i][u];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                const int line = 16 * i + 8 * u + r;
                if (j == 0) ml[warp * C::kLines + line] = make_float2(m[i][u], v);
                // columns 2 ND j .. of the line, four at a time; where they go turns with column and line (the banks)
                float *row = part + (size_t)(warp * C::kLines + line) * DP;
#pragma unroll
                for (int n = 0; n < 2 * ND; n += 4) {
                    float4 v4;
                    if (n < ND) v4 = make_float4(O[i][n][2 * u], O[i][n + 1][2 * u], O[i][n + 2][2 * u], O[i][n + 3][2 * u]);
                    else v4 = make_float4(O[i][n - ND][2 * u + 1], O[i][n - ND + 1][2 * u + 1], O[i][n - ND + 2][2 * u + 1], O[i][n - ND + 3][2 * u + 1]);
                    const int chunk = j * (ND / 2) + n / 4;
                    *reinterpret_cast<float4 *>(row + 4 * ((chunk & ~7) | ((chunk + 2 * (chunk >> 3) + line) & 7))) = v4;
                }
            }
        Piece y;
        y.r = -1;
        ok = ok && next_piece(y);
        if (meet(32 * C::NW, !ok)) return;
        {
            const int h = x.head / p.subs, sub = x.head - h * p.subs;
            const int head0 = h * p.G + sub * p.heads, heads = min(p.heads, p.G - sub * p.heads);
            const bool whole = x.slot < 0;
            constexpr int kChunks = DP / 4;
            for (int i = threadIdx.x; i < x.n * p.heads * kChunks; i += 32 * C::NW) {
                const int line = i / kChunks, chunk = i % kChunks, jj = line / p.heads, g = line - jj * p.heads;
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int w = 0; w < C::NW; ++w) M = fmaxf(M, ml[w * C::kLines + line].x);
                const float ref = M == -INFINITY ? 0.f : M;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                const int place = 4 * ((chunk & ~7) | ((chunk + 2 * (chunk >> 3) + line) & 7));
#pragma unroll
                for (int w = 0; w < C::NW; ++w) {
                    const float2 v = ml[w * C::kLines + line];
                    const float f = ex2(v.x - ref);
                    const float4 o = *reinterpret_cast<const float4 *>(part + (size_t)(w * C::kLines + line) * DP + place);
                    L = fmaf(f, v.y, L);
                    sum.x = fmaf(f, o.x, sum.x), sum.y = fmaf(f, o.y, sum.y), sum.z = fmaf(f, o.z, sum.z), sum.w = fmaf(f, o.w, sum.w);
                }
                if (g >= heads) continue;
                const int d = 4 * chunk;
                const float f = (whole ? (L == 0.f ? 0.f : 1.f / L) : 1.f) * 8.f;
                sum.x *= f, sum.y *= f, sum.z *= f, sum.w *= f;
                const size_t at = (size_t)(x.row0 + x.first + jj) * a.Hq + head0 + g, to = (size_t)(whole ? 0 : x.slot) * p.lines + line;
                if (d < a.D) {
                    if (whole)
                        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at * a.D + d) =
                            make_uint2(pack(sum.x, sum.y), pack(sum.z, sum.w));
                    else
                        *reinterpret_cast<float4 *>(p.part_o + to * p.stride + d) = sum;
                }
                if (chunk == 0) {
                    if (!whole) p.part_ml[to] = make_float2(M, L);
                    else if (a.lse) a.lse[at] = lse_of(M, L);
                }
            }
        }
        if (y.r >= 0) load_queries<C>(smem, p, y);
        if (meet(32 * C::NW, false)) return;
        x = y;
    }
}

template <typename C, bool kRows16>
__global__ void __launch_bounds__(C::kThreads, 1) tree_attention4_mma(const __grid_constant__ MmaParams mp) {
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::kOffBar), *empty = full + C::NS, *queue_full = empty + C::NS,
             *queue_empty = queue_full + kQueue;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NS; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kQueue; ++i) {
            tc::mbar_init(&queue_full[i], 1);
            tc::mbar_init(&queue_empty[i], C::NW);
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    after_predecessor();
    __syncthreads();
    const Waiter wait{abort_flag, mp.p.a.err};
    if (threadIdx.x >= 32 * C::NW) produce<C>(smem, mp, wait, full, empty, queue_full, queue_empty);
    else consume<C, kRows16>(smem, mp, wait, full, empty, queue_full, queue_empty);
    __syncthreads();
}

template <typename C, bool kRows16>
cudaError_t launch_mma_as(const MmaParams &mp, int grid, cudaStream_t s) {
    static_assert(C::kSmem <= 232448, "shared memory of a CTA");
    auto kern = tree_attention4_mma<C, kRows16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_close(kern, grid, C::kThreads, C::kSmem, s, mp);
}

}  // namespace

cudaError_t launch_mma4(Params p, int grid, cudaStream_t s) {
    const dspark_tree_attention_args &a = p.a;
    p.tile_log2 = kTileLog2;
    p.small_rows = p.block_rows;
    p.small_places = p.large_places = div_by(1);
    p.page = div_by(a.page);
    p.ctas = div_by(grid);
    p.unit_cost = kMmaUnitCost;
    MmaParams mp{p, a.page & -a.page};
    if (mp.box > kStep) mp.box = kStep;
    const bool two = p.lines > 16;
    if (a.D <= 64) return two ? launch_mma_as<MmaShape<64, 2>, false>(mp, grid, s) : launch_mma_as<MmaShape<64, 1>, false>(mp, grid, s);
    if (a.D % 32 == 0) return two ? launch_mma_as<MmaShape<128, 2>, true>(mp, grid, s) : launch_mma_as<MmaShape<128, 1>, true>(mp, grid, s);
    return two ? launch_mma_as<MmaShape<128, 2>, false>(mp, grid, s) : launch_mma_as<MmaShape<128, 1>, false>(mp, grid, s);
}

}  // namespace attn
}  // namespace dspark
