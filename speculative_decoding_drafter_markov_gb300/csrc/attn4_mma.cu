// attn4_mma.cu -- attention of few lines over a cache in 4 bits: values unpacked in
// registers, products by the warp's own matrix instructions.
//
// While a unit has few lines the cache is read for few products, and what counts is how
// a tile gets from 4 bits to the tensor cores.  Through shared memory as 16-bit tiles (the
// kernel of attn4_tc.cu) a tile of 128 tokens is written and read back as 64 KB, and its two
// products take 128 rows however few are in use.  Here nothing of it goes back to
// shared memory: the fragments of an m16n8k16 product are unpacked where they are used.
//
// A unit's lines (rows x query heads of a group) are NT times 8, the columns of the products;
// their rows are tokens, and then columns of values.  One warp walks the CTA's
// share of the work and hands out its pieces; warp w of the NW others takes every NW-th step
// of 32 tokens, with a running maximum and sum and 8 NT x D sums of its own, and the warps'
// results are added at the piece's end like partials.  A warp copies its steps itself, by
// cp.async into slots of its own, the next ones while it works on one, on into the next
// piece.  (Bulk copies by one warp took 80 clocks each to issue, 1900 to 2600 a tile: more
// than all the rest.)  Per step and warp:
//     S^T = K Q^T        K in bf16 (exactly), contracted over D in an order of its own:
//                        lane j of four has columns j D/4 .. of a token, 16 adjacent bytes
//     P = 2^(S scale log2(e) - m), rounded to fp16; m moves when a weight would pass 2^15
//     O^T += V^T P^T     V in fp16 as eighths (exactly); lane r of eight has the D / 8 columns
//                        from r D/8 on, two of them rows r and r + 8 of each product
// The 16 rows of a product are tokens in the order 0 4 1 5 2 6 3 7, 8 12 .., so that the tokens
// whose values four lanes read are adjacent, and both reads are free of bank conflicts.  P^T
// comes from S^T's fragments by an 8 x 8 transposition in the warp.
//
// What bounds it are the instructions that unpack: per two elements a mask with an
// exponent (half rate), 3/4 of a shift for keys, 1/4 and as many byte permutations for values, and
// one (keys) or two (values) fp16 operations, all of half the rate of fp32; 32 NT matrix products of 8 clocks.
#include "attn_tc_kernel.cuh"

namespace dspark {
namespace attn {

namespace {

constexpr int kStep = 32;     // tokens of a step
constexpr float kLift = 7.f;  // the reference stands below the maximum, as in attn_tc_kernel.cuh
constexpr int kMmaUnitCost = 4;

// DP: D padded, NT: lines / 8, FULL: D is DP
template <int DP_, int NT_, bool FULL_>
struct MmaShape {
    static constexpr int DP = DP_, NT = NT_;
    static constexpr bool FULL = FULL_;
    // with the walker 16 warps of 128 registers, 12 of 168 or 8 of 255
    static constexpr int NW = NT == 1 ? 15 : NT == 2 ? 11 : 7, kThreads = 32 * (NW + 1);
    static constexpr int kLines = 8 * NT;
    static constexpr int kDepth = NT < 4 ? 2 : 3;       // slots of a warp, a step each
    static constexpr int kSlot = kStep * DP / 16 * 18;  // codes of keys, of values, scales of keys, of values
    static constexpr int kOffO = NW * kDepth * kSlot;   // float [NW][kLines][DP]
    static constexpr int kOffQ = kOffO + NW * kLines * DP * 4;  // uint2 [DP / 16][32][NT]
    static constexpr int kOffMl = kOffQ + NT * DP / 16 * 256;   // float2 [NW][kLines]
    static constexpr int kOffPiece = kOffMl + NW * kLines * 8;
    static constexpr int kOffBar = kOffPiece + 64 * kQueue;
    static constexpr int kOffMisc = kOffBar + 8 * (2 * kQueue);
    static constexpr int kSmem = kOffMisc + 8;
    static_assert(kSlot % 16 == 0 && kOffPiece % 16 == 0, "places");
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], const uint2 &b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint2 &b) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
// an 8 x 8 matrix of 16-bit elements, lane 4 r + j with elements 2 j and 2 j + 1 of row r, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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

// steps of a piece
__device__ __forceinline__ int steps_of(const Piece &x) {
    return (min(x.t1 << kTileLog2, x.tokens) - (x.t0 << kTileLog2) + kStep - 1) / kStep;
}

// ---------------------------------------------------------------- the walk
template <typename C>
__device__ __forceinline__ void hand_out(unsigned char *smem, const Params &p, const Waiter &wait, uint64_t *queue_full, uint64_t *queue_empty) {
    const int lane = threadIdx.x & 31;
    const Share share = share_of(p);
    Walk walk(p, share);
    if (lane == 0) p.join[blockIdx.x].pieces = 0;
    Piece x;
    bool more = true;
    for (uint32_t k = 0; more; ++k) {
        more = walk.next(x);
        if (!more) x.r = -1;
        const int i = k % kQueue;
        if (!wait.warp(&queue_empty[i], ((k / kQueue) & 1u) ^ 1u)) break;
        if (lane == 0) {
            *reinterpret_cast<Piece *>(smem + C::kOffPiece + 64 * i) = x;
            tc::mbar_arrive(&queue_full[i]);
            if (more && x.t0 == 0 && x.t1 < x.tiles) p.join[blockIdx.x] = walk.join_of(x);
        }
    }
}

// ---------------------------------------------------------------- a warp's copies
// Position of the next step to copy: of piece `piece` (counted over the CTA's pieces), step
// s; the pages of its four groups of eight tokens (lane % 4) are fetched a step ahead.
template <typename C>
struct Copies {
    int piece, s, steps;   // s >= steps: none is left in the piece
    uint32_t c0;           // the CTA's steps before the piece
    int tok0, last;        // first token of the step; the unit's last one
    int page, off;         // of this lane's group: page, token in it
    int h;                 // key-value head
    bool more;             // a piece follows
    uint32_t issued, used;

    __device__ __forceinline__ bool any() const { return s < steps; }
};
__device__ __forceinline__ void cp_async8(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}

// ---------------------------------------------------------------- the consumers
// the queries of a unit as fragments of the first product, zero beyond its lines and columns
template <typename C>
__device__ __forceinline__ void load_queries(unsigned char *smem, const Params &p, const Piece &x) {
    constexpr int kParts = C::DP / 4, kLane = C::DP / 4;  // parts of 4 elements of a line; columns of a lane
    const dspark_tree_attention_args &a = p.a;
    const int h = x.head / p.subs, sub = x.head - h * p.subs;
    const int head0 = h * p.G + sub * p.heads, heads = min(p.heads, p.G - sub * p.heads);
    uint2 *q = reinterpret_cast<uint2 *>(smem + C::kOffQ);
    for (int i = threadIdx.x; i < C::kLines * kParts; i += 32 * C::NW) {
        const int line = i / kParts, d = (i % kParts) * 4, jj = line / p.heads, g = line - jj * p.heads;
        uint2 v = make_uint2(0u, 0u);
        if (jj < x.n && g < heads && d < a.D)
            v = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.q) + (long long)(x.row0 + x.first + jj) * a.q_row +
                                                 (head0 + g) * a.q_head + d);
        const int j = d / kLane, ks = (d % kLane) / 4;
        q[(ks * 32 + (line & 7) * 4 + j) * C::NT + (line >> 3)] = v;
    }
}

template <typename C>
__device__ __forceinline__ void consume(unsigned char *smem, const Params &p, const Waiter &wait, uint64_t *queue_full, uint64_t *queue_empty) {
    constexpr int DP = C::DP, NT = C::NT, KS = DP / 16, MT = DP / 16, ND = DP / 8;  // steps of the first product, rows / 16 of the second, columns of a lane
    const dspark_tree_attention_args &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    const int code_row = a.D / 2, scale_row = a.D / 16;
    const float scale = fmaxf(p.scale_log2, 1e-37f);  // 0 would make -inf x 0 of what is not seen
    const int token_r = (r >> 1) + 4 * (r & 1);  // token of a product's row r; of row r + 8 eight on
    const uint2 *q = reinterpret_cast<const uint2 *>(smem + C::kOffQ) + lane * NT;
    float *part = reinterpret_cast<float *>(smem + C::kOffO);
    float2 *ml = reinterpret_cast<float2 *>(smem + C::kOffMl);
    unsigned char *slots = smem + warp * (C::kDepth * C::kSlot);
    auto piece_at = [&](int i) -> const Piece & { return *reinterpret_cast<const Piece *>(smem + C::kOffPiece + 64 * (i % kQueue)); };
    auto wait_piece = [&](int i) { return wait.warp(&queue_full[i % kQueue], ((uint32_t)i / kQueue) & 1u); };
    bool ok = true;
    int now = 0;      // the piece being worked on
    Copies<C> cp{-1, 0, 0, 0, 0, 0, 0, 0, 0, true, 0, 0};
    // to the next step of this warp, in the piece being worked on or the one after it, and its pages
    auto seek = [&]() {
        while (!cp.any() && cp.more && cp.piece <= now && ok) {
            cp.c0 += (uint32_t)cp.steps;
            ++cp.piece;
            ok = wait_piece(cp.piece);
            if (!ok) break;
            const Piece &y = piece_at(cp.piece);
            cp.more = y.r >= 0;
            cp.steps = cp.more ? steps_of(y) : 0;
            cp.s = (warp + C::NW - cp.c0 % C::NW) % C::NW;
        }
        if (!cp.any()) return;
        const Piece &y = piece_at(cp.piece);
        cp.last = y.tokens - 1;
        cp.tok0 = (y.t0 << kTileLog2) + cp.s * kStep;
        cp.h = p.subs == 1 ? y.head : y.head / p.subs;
        const int tok = min(cp.tok0 + 8 * j, cp.last & ~7), in_table = p.page.of(tok);
        cp.off = tok - in_table * a.page;
        cp.page = a.table[(size_t)y.r * a.max_pages + in_table];
    };
    const long long page_bytes = cache4::page_bytes(a.page, a.D), codes = cache4::code_bytes(a.page, a.D);
    auto copy = [&]() {
        unsigned char *to = slots + (cp.issued % C::kDepth) * C::kSlot;
        int page = cp.page;
        if (page < 0 || page >= a.n_pages) {
            set_err(a.err, DSPARK_ERR_RANGE);
            page = 0;
        }
        const long long at = ((long long)page * a.H + cp.h) * page_bytes;
        const unsigned char *kc = static_cast<const unsigned char *>(a.k_cache), *vc = static_cast<const unsigned char *>(a.v_cache);
        // eight tokens' codes are adjacent, 4 D bytes, and so are their scales, D / 2
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const long long from = __shfl_sync(0xffffffffu, at + (long long)cp.off * code_row, g) + 16 * lane;
            if (cp.tok0 + 8 * g <= cp.last && 4 * lane < a.D) {
                unsigned char *dst = to + 8 * g * code_row + 16 * lane;
                cp_async16(dst, kc + from);
                cp_async16(dst + kStep * code_row, vc + from);
            }
        }
        const int g = lane >> 3, e = lane & 7;
        const long long from = __shfl_sync(0xffffffffu, at + codes + (long long)cp.off * scale_row, g) + 8 * e;
        if (cp.tok0 + 8 * g <= cp.last && 16 * e < a.D) {
            unsigned char *dst = to + 2 * kStep * code_row + 8 * g * scale_row + 8 * e;
            cp_async8(dst, kc + from);
            cp_async8(dst + kStep * scale_row, vc + from);
        }
        tc::cp_async_commit();
        ++cp.issued;
        cp.s += C::NW;
        seek();
    };
    auto fill = [&]() {
        while (cp.any() && cp.issued - cp.used < (uint32_t)C::kDepth) copy();
    };
    seek();
    Piece x;
    x.r = -1;
    if (ok) x = piece_at(0);
    if (x.r >= 0) {
        fill();
        load_queries<C>(smem, p, x);
    }
    if (meet(32 * C::NW, !ok)) {
        tc::cp_async_wait<0>();
        return;
    }
    uint32_t c0 = 0;  // steps before the piece
    while (x.r >= 0) {
        const int steps = steps_of(x);
        fill();
        const int base_rel = a.mask ? 0 : x.first + 1;  // rows of the cycle before it are seen by every line
        // lines 2 j, 2 j + 1 (+ 8 i); columns r ND + 2 t, r ND + 2 t + 1
        float O[NT][MT][4];
        float2 m[NT], l[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) O[i][t][e] = 0.f;
            m[i] = make_float2(-INFINITY, -INFINITY);
            l[i] = make_float2(0.f, 0.f);
        }
        uint2 q_held[NT == 1 ? KS : 1];
        if (NT == 1) {
#pragma unroll
            for (int k = 0; k < (NT == 1 ? KS : 0); ++k) q_held[k] = q[k * 32];
        }
        const uint32_t skip = (warp + C::NW - c0 % C::NW) % C::NW;
#pragma unroll 1
        for (int s = skip; s < steps; s += C::NW) {
            int tok0 = (x.t0 << kTileLog2) + s * kStep;
            // copies of this step: the oldest; all but it may be under way where the slots are full
            if (cp.issued - cp.used == (uint32_t)C::kDepth) tc::cp_async_wait<C::kDepth - 1>();
            else tc::cp_async_wait<0>();
            __syncwarp();
            const unsigned char *kcode = slots + (cp.used % C::kDepth) * C::kSlot, *vcode = kcode + kStep * code_row,
                                *kscale = vcode + kStep * code_row, *vscale = kscale + kStep * scale_row;
            const bool tail = tok0 + kStep > x.len + base_rel;
            // 16 tokens at a time, in a loop: its code has to stay in the first instruction cache
#pragma unroll 1
            for (int t = 0; t < 2; ++t, tok0 += 16, kcode += 16 * code_row, vcode += 16 * code_row, kscale += 16 * scale_row, vscale += 16 * scale_row) {
            // ------------------------------------------------ S^T = K Q^T
            float S[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[i][e] = 0.f;
            {
                uint32_t kw[2][KS / 2], ks[2][KS / 4], koff[2][KS / 4];
                uint32_t bytes[2][KS / 4], most = 0;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int tok = 8 * u + token_r;
                    const unsigned char *at = kcode + tok * code_row + j * (DP / 8), *sc = kscale + tok * scale_row + j * (DP / 64);
                    if (C::FULL && DP == 128) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(at);
                        kw[u][0] = w.x, kw[u][1] = w.y, kw[u][KS / 2 - 2] = w.z, kw[u][KS / 2 - 1] = w.w;
                    } else {
#pragma unroll
                        for (int g = 0; g < KS / 4; ++g) {
                            uint2 w = make_uint2(0u, 0u);
                            if (C::FULL || j * (DP / 4) + 16 * g < a.D) w = *reinterpret_cast<const uint2 *>(at + 8 * g);
                            kw[u][2 * g] = w.x, kw[u][2 * g + 1] = w.y;
                        }
                    }
#pragma unroll
                    for (int g = 0; g < KS / 4; ++g) {
                        const bool in = C::FULL || j * (DP / 4) + 16 * g < a.D;
                        bytes[u][g] = in ? sc[g] : 0u;
                        most = max(most, bytes[u][g]);
                        ks[u][g] = cache4::bf16_scales(bytes[u][g]);
                    }
                }
                if (most == cache4::kNoNumbers) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int g = 0; g < KS / 4; ++g)
                            if (bytes[u][g] == cache4::kNoNumbers) ks[u][g] = 0x7fc07fc0u;
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int g = 0; g < KS / 4; ++g)
                        koff[u][g] = cache4::bf16_offset(ks[u][g]);
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const int w = k >> 1, p0 = 2 * (k & 1), g = k >> 2;
                    const uint32_t ka[4] = {cache4::bf16_of(kw[0][w], p0, ks[0][g], koff[0][g]), cache4::bf16_of(kw[1][w], p0, ks[1][g], koff[1][g]),
                                            cache4::bf16_of(kw[0][w], p0 + 1, ks[0][g], koff[0][g]), cache4::bf16_of(kw[1][w], p0 + 1, ks[1][g], koff[1][g])};
                    if (NT == 1) {
                        mma_bf16(S[0], ka, q_held[NT == 1 ? k : 0]);
                    } else {
#pragma unroll
                        for (int i = 0; i < NT; i += 2) {
                            const uint4 two = *reinterpret_cast<const uint4 *>(q + k * 32 * NT + i);
                            mma_bf16(S[i], ka, make_uint2(two.x, two.y));
                            mma_bf16(S[NT == 1 ? 0 : i + 1], ka, make_uint2(two.z, two.w));
                        }
                    }
                }
            }
            // ------------------------------------------------ the values' words, and the slot is free
            uint32_t vw[4][ND / 8], vs[4], v_most = 0;
            {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int tok = 4 * e + j;
                    const bool in = C::FULL || r * ND < a.D;
                    const unsigned char *at = vcode + tok * code_row + r * (ND / 2);
                    if (DP == 128) {
                        uint2 w = make_uint2(0u, 0u);
                        if (in) w = *reinterpret_cast<const uint2 *>(at);
                        vw[e][0] = w.x, vw[e][ND / 8 - 1] = w.y;
                    } else {
                        vw[e][0] = in ? *reinterpret_cast<const uint32_t *>(at) : 0u;
                    }
                    vs[e] = in ? vscale[tok * scale_row + r * ND / 16] : 0u;
                    v_most = max(v_most, vs[e]);
                }
            }
            uint32_t no_numbers = 0u;  // tokens of this step whose scale of columns r ND .. is NaN for those who see them
            if (tail) {
                // what some lines do not see must not reach them as 0 x NaN: it counts as zeros here, and
                // the lines that do see it are told below
#pragma unroll 1
                for (int i = 0; i < 16; ++i) {
                    const int rel = tok0 + i - x.len;
                    if (rel < base_rel || tok0 + i >= x.tokens || r * ND >= a.D) continue;
                    if (vscale[i * scale_row + r * ND / 16] == cache4::kNoNumbers) no_numbers |= 1u << i;
                }
            }
            if (t) {
                __syncwarp();
                ++cp.used;
                if (cp.any()) copy();
            }
            // ------------------------------------------------ the weights
            uint32_t see[NT][2];
            if (tail) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int line = 8 * i + 2 * j + u, jj = line / p.heads, row = x.first + jj;
                        see[i][u] = 0;
                        if (jj < x.n) {
                            const uint32_t *words = a.mask ? reinterpret_cast<const uint32_t *>(a.mask + (size_t)(x.row0 + row) * a.W) : nullptr;
                            see[i][u] = seen_bits(words, 2 * a.W, tok0 - x.len, x.rows, row);
                        }
                    }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((see[i][e & 1] >> (8 * (e >> 1) + token_r)) & 1u)) S[i][e] = -INFINITY;
            }
            float2 top[NT];
            bool over = false;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                top[i].x = fmaxf(S[i][0], S[i][2]) * scale;
                top[i].y = fmaxf(S[i][1], S[i][3]) * scale;
                over |= top[i].x > m[i].x + (kLift + kSlack) || top[i].y > m[i].y + (kLift + kSlack);
            }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    float2 v = top[i], f;
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        v.x = fmaxf(v.x, __shfl_xor_sync(0xffffffffu, v.x, d));
                        v.y = fmaxf(v.y, __shfl_xor_sync(0xffffffffu, v.y, d));
                    }
                    const float2 to = make_float2(v.x > m[i].x + (kLift + kSlack) ? v.x - kLift : m[i].x,
                                                  v.y > m[i].y + (kLift + kSlack) ? v.y - kLift : m[i].y);
                    f.x = to.x == -INFINITY ? 1.f : ex2(m[i].x - to.x);
                    f.y = to.y == -INFINITY ? 1.f : ex2(m[i].y - to.y);
                    m[i] = to;
                    l[i].x *= f.x;
                    l[i].y *= f.y;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        O[i][t][0] *= f.x, O[i][t][1] *= f.y;
                        O[i][t][2] *= f.x, O[i][t][3] *= f.y;
                    }
                }
            }
            uint2 P[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const float2 by = {scale, scale}, off = {m[i].x == -INFINITY ? 0.f : -m[i].x, m[i].y == -INFINITY ? 0.f : -m[i].y};
                const float2 a0 = fma2({S[i][0], S[i][1]}, by, off), a1 = fma2({S[i][2], S[i][3]}, by, off);
                const float2 e0 = {ex2(a0.x), ex2(a0.y)}, e1 = {ex2(a1.x), ex2(a1.y)};
                l[i] = add2(l[i], add2(e0, e1));
                P[i] = make_uint2(transpose8(pack_half(e0.x, e0.y)), transpose8(pack_half(e1.x, e1.y)));
            }
            // ------------------------------------------------ O^T += V^T P^T
            {
                uint32_t sv[2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) f[e] = cache4::eighth_of(vs[2 * half + e]);
                    if (tail || v_most == cache4::kNoNumbers) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int tok = tok0 + 8 * half + 4 * e + j;
                            const bool bad = vs[2 * half + e] == cache4::kNoNumbers;
                            if (tail && (tok >= x.tokens || (bad && tok - x.len >= base_rel))) f[e] = 0.f;
                            else if (bad) f[e] = NAN;
                        }
                    }
                    sv[half] = pack_half(f[0], f[1]);
                }
#pragma unroll
                for (int w = 0; w < ND / 8; ++w) {
                    // the elements of even and of odd places of two tokens side by side, for either half of the 16
                    uint32_t two[2][2];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        two[half][0] = __byte_perm(vw[2 * half][w], vw[2 * half + 1][w], 0x5410);
                        two[half][1] = __byte_perm(vw[2 * half][w], vw[2 * half + 1][w], 0x7632);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int sh = 8 * (e >> 1), odd = e & 1;
                        const uint32_t va[4] = {cache4::half_of(two[0][0] >> sh, odd, sv[0]), cache4::half_of(two[0][1] >> sh, odd, sv[0]),
                                                cache4::half_of(two[1][0] >> sh, odd, sv[1]), cache4::half_of(two[1][1] >> sh, odd, sv[1])};
#pragma unroll
                        for (int i = 0; i < NT; ++i) mma_f16(O[i][4 * w + e], va, P[i]);
                    }
                }
            }
            if (tail && no_numbers) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (see[i][e & 1] & no_numbers) {
#pragma unroll
                            for (int t = 0; t < MT; ++t) O[i][t][e] = NAN;
                        }
            }
            }
        }
        c0 += (uint32_t)steps;

        // ---------------------------------------------------- the piece's end
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float2 v = l[i];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
                v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
                v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int line = 8 * i + 2 * j + u;
                if (r == 0) ml[warp * C::kLines + line] = make_float2(u ? m[i].y : m[i].x, u ? v.y : v.x);
                // columns ND r .. of the line, four at a time; where they go turns with the line (the banks)
                float *row = part + (size_t)(warp * C::kLines + line) * DP;
#pragma unroll
                for (int n = 0; n < ND; n += 4) {
                    const int chunk = r * (ND / 4) + n / 4;
                    *reinterpret_cast<float4 *>(row + 4 * ((chunk & ~7) | ((chunk + (line >> 1)) & 7))) =
                        make_float4(O[i][n / 2][u], O[i][n / 2][2 + u], O[i][n / 2 + 1][u], O[i][n / 2 + 1][2 + u]);
                }
            }
        }
        Piece y;
        y.r = -1;
        ok = ok && wait_piece(now + 1);
        if (ok) y = piece_at(now + 1);
        if (meet(32 * C::NW, !ok)) {
            tc::cp_async_wait<0>();
            return;
        }
        if (lane == 0) tc::mbar_arrive(&queue_empty[now % kQueue]);
        ++now;
        if (!cp.any()) seek();
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
                const int place = 4 * ((chunk & ~7) | ((chunk + (line >> 1)) & 7));
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

template <typename C>
__global__ void __launch_bounds__(C::kThreads, 1) tree_attention4_mma(const __grid_constant__ Params p) {
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *queue_full = reinterpret_cast<uint64_t *>(smem + C::kOffBar), *queue_empty = queue_full + kQueue;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < kQueue; ++i) {
            tc::mbar_init(&queue_full[i], 1);
            tc::mbar_init(&queue_empty[i], C::NW);
        }
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    after_predecessor();
    __syncthreads();
    const Waiter wait{abort_flag, p.a.err};
    if (threadIdx.x >= 32 * C::NW) hand_out<C>(smem, p, wait, queue_full, queue_empty);
    else consume<C>(smem, p, wait, queue_full, queue_empty);
}

template <typename C>
cudaError_t launch_mma_as(const Params &p, int grid, cudaStream_t s) {
    static_assert(C::kSmem <= 232448, "shared memory of a CTA");
    auto kern = tree_attention4_mma<C>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_close(kern, grid, C::kThreads, C::kSmem, s, p);
}

template <int DP, bool FULL>
cudaError_t launch_lines(const Params &p, int nt, int grid, cudaStream_t s) {
    return nt == 1   ? launch_mma_as<MmaShape<DP, 1, FULL>>(p, grid, s)
           : nt == 2 ? launch_mma_as<MmaShape<DP, 2, FULL>>(p, grid, s)
                     : launch_mma_as<MmaShape<DP, 4, FULL>>(p, grid, s);
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
    const int nt = p.lines <= 8 ? 1 : p.lines <= 16 ? 2 : 4;
    if (a.D == 128) return launch_lines<128, true>(p, nt, grid, s);
    if (a.D == 64) return launch_lines<64, true>(p, nt, grid, s);
    return a.D > 64 ? launch_lines<128, false>(p, nt, grid, s) : launch_lines<64, false>(p, nt, grid, s);
}

}  // namespace attn
}  // namespace dspark
